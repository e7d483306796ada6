"""The serving kernels at the ends of their ranges, against float64 (needs a B200)."""
import pytest
import torch

from tests import serving_plain as plain
from tests.test_gpu_serving import BF16, E4M3, F32, _cache, _check_packed, _cu, _gen, _plan, _randn, _sigma, _table_of

pytestmark = pytest.mark.gpu


def _at(*xs):
    return torch.tensor(xs, dtype=torch.int32, device="cuda:0")


def _along(g, T, H, H_kv, d, score, dtype=BF16):
    """q and k whose scores lie around `score`: both along one direction of +-1, and noise (some five to either side)."""
    w = torch.sign(torch.randn(d, generator=g, device="cuda:0"))
    a = (abs(score) / d ** 0.5) ** 0.5  # q k / sqrt d = a^2 sqrt d
    q = a * w + torch.randn((T, H, d), generator=g, device="cuda:0")
    k = (a if score > 0 else -a) * w + torch.randn((T, H_kv, d), generator=g, device="cuda:0")
    return q.to(dtype), k.to(dtype)


def _check_chunks(plan, cache, pt, q, ends, chunks, max_new=None):
    """The last chunks[n] of ends[n] tokens of every sequence (packed in q) against what the cache holds; q holds all tokens."""
    zero = _at(*[0] * len(ends))
    K, V = (x.double() for x in cache.read(pt, _cu(ends), zero, sum(ends), dtype=F32 if cache.quantised else cache.dtype))
    first = [sum(ends[:n]) for n in range(len(ends))]
    new = torch.cat([q[a + e - c:a + e] for a, e, c in zip(first, ends, chunks)])
    O, R = plan.attend_paged(new, cache, pt, _cu(chunks), _at(*[e - c for e, c in zip(ends, chunks)]), max_new=max_new)
    plan.check()
    cache.check()
    t = 0
    for n, (a, e, c) in enumerate(zip(first, ends, chunks)):
        want = plain.sequence(new[t:t + c].double(), K[a:a + e], V[a:a + e], plan.table_host, e - c)
        plain.check(O[t:t + c], R[t:t + c], want, plan.dtype, f"sequence {n}, {c} of {e} tokens")
        t += c


@pytest.mark.parametrize("score", [-80.0, -100.0, -150.0, -400.0])
@pytest.mark.parametrize("d,kind", [(128, E4M3), (128, BF16), (64, E4M3), (64, BF16)])
def test_rows_whose_scores_all_lie_far_below_zero(d, kind, score):
    """A shift of all of a row's scores leaves its weights as they are: prompts, chunks and single tokens."""
    H, H_kv, lens = 4, 2, [33, 64, 100, 129, 300]
    T, g = sum(lens), _gen(70)
    plan = _plan(H, H_kv, 320, d, 20, BF16, sigma=[1.0, 20.0, 90.0, 2000.0])
    q, k = _along(g, T, H, H_kv, d, score)
    v = _randn(g, T, H_kv, d)
    O, R = plan.attend_packed(q, k, v, _cu(lens))
    plan.check()
    _check_packed(plan, O, R, q, k, v, lens)
    pt, num = _table_of(lens, 32)
    cache = _cache(num, H_kv, 32, d, kind)
    cache.append(k, v, pt, _cu(lens), _at(*[0] * len(lens)))
    _check_chunks(plan, cache, pt, q, lens, [33, 40, 70, 100, 150])
    _check_chunks(plan, cache, pt, q, lens, [1] * 5, max_new=1)

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


def _shifted(x):
    """A copy of x 16 bytes into a larger buffer: aligned to 16 bytes and to no more."""
    n = 16 // x.element_size()
    y = torch.empty(x.numel() + n, dtype=x.dtype, device=x.device)[n:].view(x.shape)
    assert y.data_ptr() % 32 == 16
    return y.copy_(x)


@pytest.mark.parametrize("d,dtype", [(128, BF16), (64, BF16), (64, F32)])
def test_tensors_aligned_to_16_bytes(d, dtype):
    import alibi_positional_lsh_b200 as m
    H, H_kv, s, page, lens = 4, 2, 20, 32, [200, 1, 77, 130]
    T, g, n = sum(lens), _gen(71), len(lens)
    plan = _plan(H, H_kv, 210, d, s, dtype)
    q, k, v = (_randn(g, T, h, d, dtype=dtype) for h in (H, H_kv, H_kv))
    cu, zero = _cu(lens), _at(*[0] * n)
    sq, sk, sv = _shifted(q), _shifted(k), _shifted(v)
    out = _shifted(torch.zeros_like(q)), _shifted(torch.zeros((T, H), device="cuda:0"))
    want = plan.attend_packed(q, k, v, cu)
    got = plan.attend_packed(sq, sk, sv, cu, out=out)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    pt, num = _table_of(lens, page)
    for kind in (E4M3, dtype):
        a = _cache(num, H_kv, page, d, kind)
        b = m.PagedCache(*(None if x is None else _shifted(x) for x in (a.k_pages, a.v_pages, a.k_exp, a.v_exp)))
        a.append(k, v, pt, cu, zero)
        b.append(sk, sv, pt, cu, zero)
        rows = a.read(pt, cu, zero, T, dtype=dtype)
        back = b.read(pt, cu, zero, T, out=(_shifted(torch.zeros_like(k)), _shifted(torch.zeros_like(v))))
        assert all(torch.equal(x, y) for x, y in zip(rows, back))
        for most in (None, 200):
            want = plan.attend_paged(q, a, pt, cu, zero, max_new=most)
            got = plan.attend_paged(sq, b, pt, cu, zero, max_new=most, out=out)
            assert all(torch.equal(x, y) for x, y in zip(want, got))
        tok, one = _at(*[L - 1 for L in lens]), _cu([1] * n)
        want = plan.attend_paged(q[:n], a, pt, one, tok, max_new=1)
        got = plan.attend_paged(sq[:n], b, pt, one, tok, max_new=1, out=(out[0][:n], out[1][:n]))
        assert all(torch.equal(x, y) for x, y in zip(want, got))
        if kind == E4M3 and dtype == BF16:
            scratch = _shifted(torch.zeros(m.plsh_paged_scratch_bytes(T, n, T, H_kv, d, plan.max_window), dtype=torch.uint8, device="cuda:0"))
            want = plan.attend_paged(q, a, pt, cu, zero)
            err = torch.zeros(4, dtype=torch.int32, device="cuda:0")
            m.plsh_paged_fwd(q, m.PLSH_BF16, cu, zero, T, H, H_kv, d, b.k_pages, b.v_pages, b.k_exp, b.v_exp, pt, s, 210, plan.table_dev,
                             plan.spans, plan.bmask, plan.near, plan.windows_host, scratch, out[0], out[1], err)
            assert all(torch.equal(x, y) for x, y in zip(want, out)) and int(err.abs().max()) == 0
        b.check()
    plan.check()


@pytest.mark.parametrize("score", [30.0, 33.0, 36.0, 45.0])
@pytest.mark.parametrize("d,kind,dtype", [(128, E4M3, BF16), (128, BF16, BF16), (64, BF16, BF16), (64, F32, F32)])
def test_values_up_to_2_to_the_64_under_high_scores(d, kind, dtype, score):
    """A row's result is no larger than its largest value: no sum before the division may overflow."""
    H, H_kv, lens = 4, 2, [33, 70, 129, 300]
    T, g = sum(lens), _gen(72)
    plan = _plan(H, H_kv, 320, d, 20, dtype, sigma=[1.0, 20.0, 90.0, 2000.0])
    q, k = _along(g, T, H, H_kv, d, score, dtype)
    sign = torch.sign(torch.randn(d, generator=g, device="cuda:0"))  # a column's values do not cancel
    v = (sign * (1 + torch.rand((T, H_kv, d), generator=g, device="cuda:0")) * 2.0 ** 63).to(dtype)
    O, R = plan.attend_packed(q, k, v, _cu(lens))
    plan.check()
    _check_packed(plan, O, R, q, k, v, lens)
    pt, num = _table_of(lens, 32)
    cache = _cache(num, H_kv, 32, d, kind)
    cache.append(k, v, pt, _cu(lens), _at(*[0] * len(lens)))
    _check_chunks(plan, cache, pt, q, lens, [33, 40, 100, 150])
    _check_chunks(plan, cache, pt, q, lens, [1] * 4, max_new=1)


@pytest.mark.parametrize("kind,d,dtype", [(E4M3, 128, BF16), (E4M3, 64, F32), (BF16, 64, BF16), (F32, 128, F32)])
def test_rows_whose_page_is_not_there_read_as_zeros(kind, d, dtype):
    H_kv, page, lens, starts = 3, 16, [40, 1, 30], [3, 0, 20]
    T, g = sum(lens), _gen(73)
    pt, num = _table_of([a + b for a, b in zip(lens, starts)], page)
    cache = _cache(num, H_kv, page, d, kind)
    cu, st = _cu(lens), _at(*starts)
    cache.append(_randn(g, T, H_kv, d, dtype=dtype), _randn(g, T, H_kv, d, dtype=dtype), pt, cu, st)
    whole = cache.read(pt, cu, st, T, dtype=dtype)
    cache.check()
    for bad in (-1, num, 2 ** 31 - 1, -2 ** 31):
        cut = pt.clone()
        cut[0, 1], cut[2, 2] = bad, bad
        lost = torch.zeros(T + 2, dtype=torch.bool, device="cuda:0")
        for t, p, s in [(i, 3 + i, 0) for i in range(40)] + [(41 + i, 20 + i, 2) for i in range(30)]:
            lost[t] = p // page == (1 if s == 0 else 2)
        out = tuple(torch.full((T + 2, H_kv, d), 7.0, dtype=dtype, device="cuda:0") for _ in range(2))
        cache.read(cut, cu, st, T + 2, out=out)
        assert cache.device_errors() == ["PAGE"]
        cache.reset_errors()
        for x, w in zip(out, whole):
            assert (x[lost] == 0).all() and torch.equal(x[:T][~lost[:T]], w[~lost[:T]]) and (x[T:] == 7.0).all()


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 64)])
def test_plans_and_caches_keep_what_they_were_made_of(dtype, d):
    """Neither tensors nor sizes can be exchanged under the calls; deep copies have tensors of their own."""
    import copy
    H, H_kv, page, lens = 4, 2, 16, [50, 1, 70]
    T, g, zero = sum(lens), _gen(74), _at(0, 0, 0)
    plan = _plan(H, H_kv, 80, d, 20, dtype)
    pt, num = _table_of(lens, page)
    cache = _cache(num, H_kv, page, d, E4M3)
    for x, names in ((plan, "spans bmask near table_dev err windows_host max_window H H_kv d s max_len dtype device"),
                     (cache, "k_pages v_pages k_exp v_exp err num_pages H_kv page_size d dtype device quantised")):
        for name in names.split():
            with pytest.raises(AttributeError):
                setattr(x, name, getattr(x, name))
    with pytest.raises(ValueError):
        plan.windows_host[0] = 1 << 20
    q, k, v = (_randn(g, T, h, d, dtype=dtype) for h in (H, H_kv, H_kv))
    cache.append(k, v, pt, _cu(lens), zero)
    want = plan.attend_paged(q, cache, pt, _cu(lens), zero) + plan.attend_packed(q, k, v, _cu(lens))
    plan2, cache2 = copy.deepcopy(plan), copy.deepcopy(cache)
    for t in (cache.k_pages, cache.v_pages):  # the first cache's rows go, the copy's stay
        t.view(torch.uint8).zero_()
    plan.spans.zero_()
    plan.near.zero_()
    got = plan2.attend_paged(q, cache2, pt, _cu(lens), zero) + plan2.attend_packed(q, k, v, _cu(lens))
    plan2.check()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def _window_start(plan, p):
    """The lowest position that shares a bin with p, of any head's hashes."""
    delta, u = (torch.tensor(plan.table_host[..., i]) for i in range(2))
    j = torch.arange(p + 1, dtype=torch.float64)
    same = torch.floor((j[:, None, None] + u) / delta) == torch.floor((p + u) / delta)
    return int(same.flatten(1).any(1).nonzero()[0])


BEHIND = [
    # kind, d, dtype, s, H, H_kv, page, sigma, lens, starts
    (E4M3, 128, BF16, 20, 4, 2, 16, [0.5, 2.0, 6.0, 15.0], [130, 40, 200, 17], [700, 641, 64, 1005]),
    (BF16, 128, BF16, 20, 4, 2, 16, [0.5, 2.0, 6.0, 15.0], [130, 40, 200, 17], [700, 641, 64, 1005]),
    (BF16, 64, BF16, 20, 4, 2, 32, [0.5, 1.0, 1.5, 2.0], [100, 64, 20, 300], [703, 704, 767, 768]),
    (BF16, 128, BF16, 40, 4, 1, 16, [0.5, 1.0, 9.0, 30.0], [33, 18, 129], [415, 831, 640]),
    (E4M3, 64, BF16, 33, 6, 2, 64, [1.0, 1.0, 2.0, 20.0, 30.0, 30.0], [18, 140, 64], [900, 640, 1023]),
    (BF16, 64, BF16, 20, 2, 2, 256, [1.0, 20.0], [30, 260], [900, 600]),
    (E4M3, 128, BF16, 20, 8, 2, 16, [0.5, 1.0, 2.0, 2.0, 3.0, 3.0, 9.0, 30.0], [1, 3, 8, 1, 2], [900, 641, 64, 63, 400]),
    (BF16, 64, BF16, 20, 4, 2, 32, [0.5, 1.0, 2.0, 15.0], [1, 3, 8, 1, 16], [900, 641, 64, 63, 400]),
    (F32, 64, F32, 20, 4, 2, 16, [0.5, 2.0, 6.0, 15.0], [1, 100, 33, 64], [700, 641, 96, 1005]),
    (E4M3, 128, BF16, 20, 2, 1, 16, [1.0, 9.0], [20, 33], [800, 927]),   # in the plan's last row tile
    (E4M3, 128, F32, 40, 2, 1, 32, [1.0, 3.0], [1, 70, 5], [703, 704, 767]),
    (F32, 64, F32, 20, 16, 4, 16, [0.5 + 0.5 * h for h in range(16)], [600, 500, 700, 550, 640], [701, 640, 96, 1005, 32]),
]


@pytest.mark.parametrize("kind,d,dtype,s,H,H_kv,page,sigma,lens,starts", BEHIND, ids=[str(n) for n in range(len(BEHIND))])
def test_pages_behind_the_window_may_be_anything(kind, d, dtype, s, H, H_kv, page, sigma, lens, starts):
    """A server hands on pages that no later token reaches: entries then name nothing, or another sequence's page."""
    ends = [a + b for a, b in zip(lens, starts)]
    plan, g = _plan(H, H_kv, max(ends) + 5, d, s, dtype, sigma=sigma), _gen(75)
    pt, num = _table_of(ends, page, spare=3)
    cache = _cache(num, H_kv, page, d, kind)   # pages without an owner hold NaN
    T = sum(ends)
    cache.append(_randn(g, T, H_kv, d, dtype=dtype), _randn(g, T, H_kv, d, dtype=dtype), pt, _cu(ends), _at(*[0] * len(ends)))
    K, V = (x.double() for x in cache.read(pt, _cu(ends), _at(*[0] * len(ends)), T, dtype=F32 if cache.quantised else dtype))
    unowned = [n for n in range(num) if not (pt == n).any()]
    lost = [_window_start(plan, a) // page for a in starts]
    assert sum(lost) >= 4
    q, cu, st = _randn(g, sum(lens), H, d, dtype=dtype), _cu(lens), _at(*starts)
    for most in (max(lens), None):
        want = plan.attend_paged(q, cache, pt, cu, st, max_new=most)
        plan.check()
        t = at = 0
        for n, (L, a) in enumerate(zip(lens, starts)):
            full = plain.sequence(q[t:t + L].double(), K[at:at + a + L], V[at:at + a + L], plan.table_host, a)
            plain.check(want[0][t:t + L], want[1][t:t + L], full, dtype, f"sequence {n}")
            t, at = t + L, at + ends[n]
        for entry in (-1, num, -2 ** 31, unowned[0]):
            cut = pt.clone()
            for n, c in enumerate(lost):
                cut[n, :c] = entry
            got = plan.attend_paged(q, cache, cut, cu, st, max_new=most)
            plan.check()
            assert all(torch.equal(a, b) for a, b in zip(want, got)), entry
        for n, c in enumerate(lost):  # one page more is needed
            cut = pt.clone()
            cut[n, c] = -1
            plan.attend_paged(q, cache, cut, cu, st, max_new=most)
            assert plan.device_errors() == ["PAGE"], n
            plan.reset_errors()


def test_many_sequences_under_heads_that_reach_far():
    """More windows than the scratch holds at a time: three groups of sequences, empty and single-token ones among them."""
    import alibi_positional_lsh_b200 as m
    H, H_kv, d, page, S = 8, 8, 128, 64, 40
    lens = [(17 + 3 * n) % 45 + 1 if n % 4 else n % 8 for n in range(S)]
    lens[16] = lens[31] = 140
    starts = [(37 * n) % 300 for n in range(S)]
    ends = [a + b if b else 0 for a, b in zip(starts, lens)]
    plan, g = _plan(H, H_kv, 32768, d, 20, BF16, sigma=[20000.0 + 1000 * h for h in range(H)]), _gen(76)
    assert m.plsh_paged_scratch_bytes(sum(lens), S, 140, H_kv, d, plan.max_window) < S / 2 * 4 * H_kv * d * plan.max_window
    pt, num = _table_of(ends, page)
    cache = _cache(num, H_kv, page, d, E4M3)
    T = sum(ends)
    cache.append(_randn(g, T, H_kv, d), _randn(g, T, H_kv, d), pt, _cu(ends), _at(*[0] * S))
    K, V = (x.double() for x in cache.read(pt, _cu(ends), _at(*[0] * S), T, dtype=F32))
    q = _randn(g, sum(lens), H, d)
    O, R = plan.attend_paged(q, cache, pt, _cu(lens), _at(*starts), max_new=140)
    plan.check()
    cache.check()
    t = at = 0
    for n, (L, a) in enumerate(zip(lens, starts)):
        if L:
            want = plain.sequence(q[t:t + L].double(), K[at:at + a + L], V[at:at + a + L], plan.table_host, a)
            plain.check(O[t:t + L], R[t:t + L], want, BF16, f"sequence {n}")
        t, at = t + L, at + ends[n]
    # a page missing, and a sequence too long, in the last group
    cut = pt.clone()
    last = max(n for n in range(S) if lens[n] > 17)
    cut[last, 0] = -1
    plan.attend_paged(q, cache, cut, _cu(lens), _at(*starts), max_new=140)
    assert plan.device_errors() == ["PAGE"]
    plan.reset_errors()
    late = list(starts)
    late[S - 1] = 32768
    plan.attend_paged(q, cache, pt, _cu(lens), _at(*late), max_new=140)
    assert plan.device_errors() == ["SEQUENCE"]
    plan.reset_errors()

"""Packed prompts, the paged cache and attention against it, against float64 (needs a B200)."""
import numpy as np
import pytest
import torch

import oracle
from tests import serving_plain as plain

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _sigma(H, top=8.0):
    return [2.0 ** (top * (h + 1) / H) for h in range(H)]


def _plan(H, H_kv, max_len, d, s, dtype, sigma=None, seed=3, **kw):
    from alibi_positional_lsh_b200 import PlshServing
    return PlshServing(H, H_kv, max_len, d, s, sigma or _sigma(H), seed, dtype, "cuda:0", **kw)


def _randn(g, *shape, dtype=BF16):
    return torch.randn(shape, generator=g, device="cuda:0", dtype=torch.float32).to(dtype)


def _cu(lens, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(lens)]), dtype=torch.int32, device="cuda:0")


def _gen(seed):
    return torch.Generator(device="cuda:0").manual_seed(seed)


def _check_packed(plan, O, R, q, k, v, lens, first=0, what=""):
    t = first
    for n, L in enumerate(lens):
        if L:
            want = plain.sequence(*(x[t:t + L].double() for x in (q, k, v)), plan.table_host, 0)
            plain.check(O[t:t + L], R[t:t + L], want, plan.dtype, f"{what} sequence {n} ({L} tokens)")
        t += L


# ---------------------------------------------------------------- packed prompts

PACKED = [
    # H, H_kv, d, s, dtype, lens
    (4, 2, 128, 20, BF16, [1]),
    (4, 2, 128, 20, BF16, [300, 0, 1, 129, 0, 128, 700]),
    (2, 2, 128, 1, BF16, [65, 64, 63, 257]),
    (6, 2, 128, 33, BF16, [511, 3, 1025]),
    (5, 1, 128, 64, BF16, [100, 1000]),
    (3, 3, 128, 32, BF16, [127, 900]),
    (4, 2, 64, 20, BF16, [300, 1, 129, 640]),
    (4, 1, 64, 40, BF16, [1, 2, 3, 777]),
    (4, 2, 64, 8, F32, [300, 0, 1, 129]),
    (2, 1, 128, 40, F32, [64, 65, 257]),
]


def _id(c):
    return f"H{c[0]}kv{c[1]}d{c[2]}s{c[3]}{'f32' if c[4] == F32 else 'bf16'}" + "-" + "_".join(map(str, c[5]))


@pytest.mark.parametrize("H,H_kv,d,s,dtype,lens", PACKED, ids=[_id(c) for c in PACKED])
def test_packed_matches_plain(H, H_kv, d, s, dtype, lens):
    plan = _plan(H, H_kv, max(lens) + 37, d, s, dtype)
    T, g = sum(lens), _gen(sum(lens))
    q, k, v = _randn(g, T, H, d, dtype=dtype), _randn(g, T, H_kv, d, dtype=dtype), _randn(g, T, H_kv, d, dtype=dtype)
    O, R = plan.attend_packed(q, k, v, _cu(lens))
    plan.check()
    _check_packed(plan, O, R, q, k, v, lens)


@pytest.mark.parametrize("d,dtype", [(128, BF16), (64, BF16), (64, F32)])
@pytest.mark.parametrize("sigma", [0.3, 3.0, 5000.0])
def test_packed_extreme_block_sizes(sigma, d, dtype):
    # tiny sigma: a row's own key is nearly all; huge sigma: blocks span the whole sequence
    lens = [900, 130, 258]
    plan = _plan(2, 1, 900, d, 20, dtype, sigma=[sigma, sigma * 1.5])
    g = _gen(7)
    q, k, v = _randn(g, 1288, 2, d, dtype=dtype), _randn(g, 1288, 1, d, dtype=dtype), _randn(g, 1288, 1, d, dtype=dtype)
    O, R = plan.attend_packed(q, k, v, _cu(lens))
    plan.check()
    _check_packed(plan, O, R, q, k, v, lens)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_packed_large_scores(dtype):
    # scores of several hundred: zero-weight keys far above the weighted ones must not matter
    lens, d = [700, 260], 128
    plan = _plan(2, 1, 700, d, 10, dtype, sigma=[4.0, 60.0])
    g = _gen(8)
    q, k, v = _randn(g, 960, 2, d) * 16, _randn(g, 960, 1, d) * 4, _randn(g, 960, 1, d)
    q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    O, R = plan.attend_packed(q, k, v, _cu(lens))
    plan.check()
    assert torch.isfinite(O).all() and torch.isfinite(R).all()
    _check_packed(plan, O, R, q, k, v, lens)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_packed_views_of_a_fused_projection_and_head_major(dtype, d):
    H, H_kv, lens = 4, 2, [200, 77, 131]
    T, g = sum(lens), _gen(9)
    plan = _plan(H, H_kv, 256, d, 20, dtype)
    qkv = _randn(g, T, H + 2 * H_kv, d, dtype=dtype)
    q, k, v = qkv[:, :H], qkv[:, H:H + H_kv], qkv[:, H + H_kv:]
    want = plan.attend_packed(q.contiguous(), k.contiguous(), v.contiguous(), _cu(lens))
    got = plan.attend_packed(q, k, v, _cu(lens))
    hm = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    major = plan.attend_packed(*hm, _cu(lens))
    plan.check()
    for a, b, c in zip(want, got, major):
        assert torch.equal(a, b) and torch.equal(a, c)
    _check_packed(plan, *want, q, k, v, lens)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 128)])
def test_packed_leaves_rows_of_no_sequence(dtype, d):
    # a batch padded in front and behind
    H, H_kv, lens, first, T = 4, 4, [130, 1, 250], 5, 512
    plan, g = _plan(H, H_kv, 256, d, 20, dtype), _gen(10)
    q, k, v = _randn(g, T, H, d, dtype=dtype), _randn(g, T, H_kv, d, dtype=dtype), _randn(g, T, H_kv, d, dtype=dtype)
    O, R = torch.full((T, H, d), 7.0, dtype=dtype, device="cuda:0"), torch.full((T, H), 9.0, device="cuda:0")
    plan.attend_packed(q, k, v, _cu(lens, first), out=(O, R))
    plan.check()
    end = first + sum(lens)
    for x, w in ((O, 7.0), (R, 9.0)):
        assert (x[:first] == w).all() and (x[end:] == w).all()
    _check_packed(plan, O, R, q, k, v, lens, first)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_packed_sequences_do_not_see_each_other(dtype, d, bad):
    # sequences of non-finite values between and behind finite ones, and in the padding
    H, H_kv, lens = 2, 1, [100, 60, 131, 129, 64]
    T, g = sum(lens) + 40, _gen(11)
    plan, cu = _plan(H, H_kv, 256, d, 20, dtype), _cu(lens)
    q, k, v = _randn(g, T, H, d, dtype=dtype), _randn(g, T, H_kv, d, dtype=dtype), _randn(g, T, H_kv, d, dtype=dtype)
    O, R = plan.attend_packed(q, k, v, cu)
    at = torch.zeros(T, dtype=torch.bool, device="cuda:0")
    at[100:160] = at[291:420] = at[sum(lens):] = True
    for x in (q, k, v):
        x[at] = bad
    O2, R2 = plan.attend_packed(q, k, v, cu)
    plan.check()
    at[sum(lens):] = True
    assert torch.equal(O[~at], O2[~at]) and torch.equal(R[~at], R2[~at])
    assert torch.isfinite(O2[~at]).all()


def test_packed_equals_the_dense_forward():
    """One sequence of a packed call is a batch row of the dense plan with the same table."""
    from alibi_positional_lsh_b200 import PlshForward
    H, H_kv, n, d, s = 4, 2, 1000, 128, 20
    sigma = _sigma(H)
    dense = PlshForward(1, H, H_kv, n, d, s, True, sigma, 3, BF16, "cuda:0")
    plan, g = _plan(H, H_kv, n, d, s, BF16, sigma), _gen(12)
    q, k, v = _randn(g, n, H, d), _randn(g, n, H_kv, d), _randn(g, n, H_kv, d)
    O, R = plan.attend_packed(q, k, v, _cu([n]))
    Od, Rd = dense(*(x.transpose(0, 1)[None].contiguous() for x in (q, k, v)))
    plan.check()
    assert np.array_equal(plan.table_host, dense.table_host.numpy())
    # each within 2^-7 + 2^-11 of sum w|V| <= max|V| of the same value
    assert (O.double() - Od[0].transpose(0, 1).double()).abs().max() <= 2 * (2.0 ** -7 + 2.0 ** -11) * v.abs().max()
    assert (R - Rd[0].transpose(0, 1)).abs().max() <= 1e-3


def test_packed_against_the_oracle():
    H, H_kv, d, s, lens = 2, 1, 128, 20, [260, 75]
    plan, g = _plan(H, H_kv, 300, d, s, BF16), _gen(13)
    q, k, v = _randn(g, 335, H, d), _randn(g, 335, H_kv, d), _randn(g, 335, H_kv, d)
    O, R = plan.attend_packed(q, k, v, _cu(lens))
    plan.check()
    table = oracle.draw_table(3, _sigma(H), s)
    t = 0
    for L in lens:
        for h in range(H):
            x = [y[t:t + L, c].double().cpu().numpy() for y, c in ((q, h), (k, 0), (v, 0))]
            wO, wR = oracle.approx_attention(*x, oracle.bin_ids(table, L)[h], True)
            assert np.abs(O[t:t + L, h].double().cpu().numpy() - wO).max() <= (2.0 ** -7 + 2.0 ** -10) * np.abs(x[2]).max()
            assert np.abs(R[t:t + L, h].double().cpu().numpy() - wR).max() <= 1e-4
        t += L


# ---------------------------------------------------------------- the paged cache


def _table_of(lens, page, spare=2, seed=0):
    """A page table that scatters the sequences' pages, with garbage behind each sequence's last page."""
    counts = [max(0, -(-n // page)) for n in lens]
    perm = np.random.default_rng(seed).permutation(sum(counts) + spare)
    pt = np.full((len(lens), max(counts + [1]) + 1), -7, dtype=np.int32)
    at = 0
    for s, c in enumerate(counts):
        pt[s, :c] = perm[at:at + c]
        pt[s, c:] = 10 ** 9 if s % 2 else -7
        at += c
    return torch.tensor(pt, device="cuda:0"), sum(counts) + spare


def _cache(num_pages, H_kv, page, d, dtype):
    """A cache whose unwritten places hold NaN."""
    from alibi_positional_lsh_b200 import PagedCache
    c = PagedCache.empty(num_pages, H_kv, page, d, dtype, "cuda:0")
    for t in (c.k_pages, c.v_pages):
        if dtype == E4M3:
            t.view(torch.uint8).fill_(0x7F)
        else:
            t.fill_(float("nan"))
    for t in (c.k_exp, c.v_exp):
        if t is not None:
            t.fill_(5)
    return c


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,page", [(128, 64), (64, 16), (128, 256), (64, 32)])
def test_cache_round_trip_e4m3(dtype, d, page):
    H_kv, lens, starts = 3, [5, 0, 1, 70, 33], [0, 9, 100, 17, 250]
    T, g = sum(lens), _gen(20)
    k = torch.randn((T, H_kv, d), generator=g, device="cuda:0")
    v = torch.randn((T, H_kv, d), generator=g, device="cuda:0")
    k *= torch.exp2(torch.randint(-30, 30, (T, H_kv, 1), generator=g, device="cuda:0").float())
    k[0] = 0.0
    k[1, :, 3] = 448.0 * 2.0 ** 20       # the scale's border
    k[2, 0, 5], k[2, 1, 6], k[2, 2, 0] = float("nan"), float("inf"), -float("inf")
    k[3] = 3e38
    k[4] = 1.5e-38                        # the least exponent
    v[7, 0] = 2.0 ** -140
    v[8, 1, :4] = torch.tensor([448.0, 17.0, 19.0, 0.5 * 2.0 ** -9], device="cuda:0")  # ties
    k, v = k.to(dtype), v.to(dtype)
    pt, num = _table_of([a + b for a, b in zip(starts, lens)], page)
    cache = _cache(num, H_kv, page, d, E4M3)
    before = [x.clone() for x in (cache.k_pages.view(torch.uint8), cache.v_pages.view(torch.uint8), cache.k_exp, cache.v_exp)]
    cu, st = _cu(lens), torch.tensor(starts, dtype=torch.int32, device="cuda:0")
    cache.append(k, v, pt, cu, st)
    cache.check()
    K, V = cache.read(pt, cu, st, T, dtype=dtype)
    K32, _ = cache.read(pt, cu, st, T, dtype=F32)
    cache.check()
    written = torch.zeros((num, page), dtype=torch.bool)
    ptc = pt.cpu().numpy()
    t = 0
    for s, L in enumerate(lens):
        for i in range(L):
            p = starts[s] + i
            written[ptc[s, p // page], p % page] = True
    w = written.cuda()
    for x, pages, exps, back, b4 in ((k, cache.k_pages, cache.k_exp, K, (before[0], before[2])),
                                     (v, cache.v_pages, cache.v_exp, V, (before[1], before[3]))):
        byte, exp = plain.quantise(x.double().cpu().numpy())
        raw, ex = pages.view(torch.uint8).cpu().numpy(), exps.cpu().numpy()
        t = 0
        for s, L in enumerate(lens):
            for i in range(L):
                p = starts[s] + i
                got = raw[ptc[s, p // page], :, p % page]
                nan = (byte[t] & 0x7F) == 0x7F
                assert np.array_equal(ex[ptc[s, p // page], :, p % page], exp[t]), (s, i)
                assert np.array_equal(np.where(nan, got & 0x7F, got), np.where(nan, 0x7F, byte[t])), (s, i)
                t += 1
        want = torch.tensor(plain.values(byte, exp)).to(dtype).cuda()
        assert torch.equal(torch.nan_to_num(back, nan=-3.0), torch.nan_to_num(want, nan=-3.0))
        # nothing else was touched
        keep = ~w[:, None, :].expand(-1, H_kv, -1)
        assert torch.equal(pages.view(torch.uint8)[keep], b4[0][keep]) and torch.equal(exps[keep], b4[1][keep])
    if dtype == F32:
        assert torch.equal(torch.nan_to_num(K32, nan=-3.0), torch.nan_to_num(K, nan=-3.0))


@pytest.mark.parametrize("dtype,d,page", [(BF16, 128, 16), (F32, 64, 128)])
def test_cache_round_trip_same(dtype, d, page):
    H_kv, lens, starts = 2, [40, 1, 0, 300], [3, 0, 5, 127]
    T, g = sum(lens), _gen(21)
    kv = _randn(g, T, 2 * H_kv, d, dtype=dtype)
    k, v = kv[:, :H_kv], kv[:, H_kv:]      # views
    pt, num = _table_of([a + b for a, b in zip(starts, lens)], page)
    cache = _cache(num, H_kv, page, d, dtype)
    cu, st = _cu(lens), torch.tensor(starts, dtype=torch.int32, device="cuda:0")
    cache.append(k, v, pt, cu, st)
    out = tuple(torch.full((T + 3, H_kv, d), 4.0, dtype=dtype, device="cuda:0") for _ in range(2))
    cache.read(pt, cu, st, T + 3, out=out)
    cache.check()
    assert torch.equal(out[0][:T], k) and torch.equal(out[1][:T], v)
    assert (out[0][T:] == 4.0).all() and (out[1][T:] == 4.0).all()


# ---------------------------------------------------------------- new tokens against the cache


def _fill(cache, ends, pt, g, H_kv, d, dtype):
    """Writes every position of every sequence; returns the rows as the cache holds them, packed (float64)."""
    T = sum(ends)
    k = _randn(g, T, H_kv, d, dtype=dtype) * torch.exp(0.5 * torch.randn((T, H_kv, 1), generator=g, device="cuda:0")).to(dtype)
    v = _randn(g, T, H_kv, d, dtype=dtype)
    cu, zero = _cu(ends), torch.zeros(len(ends), dtype=torch.int32, device="cuda:0")
    cache.append(k, v, pt, cu, zero)
    cache.check()
    K, V = cache.read(pt, cu, zero, T, dtype=F32 if cache.quantised else dtype)
    if not cache.quantised:
        assert torch.equal(K, k) and torch.equal(V, v)
    return K.double(), V.double()


PAGED = [
    # H, H_kv, d, s, dtype, pages, page, lens, starts
    (4, 2, 128, 20, BF16, E4M3, 64, [1], [0]),
    (4, 2, 128, 20, BF16, E4M3, 64, [1, 1, 1, 1, 1], [0, 63, 64, 1000, 1777]),
    (8, 2, 128, 33, BF16, E4M3, 16, [1, 2, 4, 3, 0, 1], [900, 0, 17, 31, 50, 700]),
    (5, 1, 128, 20, BF16, BF16, 32, [1, 3, 1], [777, 300, 2]),
    (4, 2, 128, 20, BF16, E4M3, 64, [300, 1, 77, 128], [0, 1000, 900, 64]),
    (4, 4, 128, 20, BF16, BF16, 32, [129, 64, 500], [37, 0, 700]),
    (4, 2, 128, 64, BF16, E4M3, 256, [65, 200], [1, 511]),
    (4, 2, 64, 20, BF16, E4M3, 64, [1, 5, 100, 257], [10, 0, 700, 300]),
    (6, 2, 64, 40, BF16, BF16, 128, [1, 1], [500, 3]),
    (4, 2, 64, 8, F32, F32, 32, [1, 70, 2], [300, 100, 0]),
    (2, 1, 128, 20, F32, E4M3, 64, [1, 1, 33], [400, 0, 65]),
    (16, 1, 128, 20, BF16, E4M3, 64, [1, 2], [1000, 333]),
]


def _pid(c):
    name = {BF16: "bf16", F32: "f32", E4M3: "e4m3"}
    return f"H{c[0]}kv{c[1]}d{c[2]}s{c[3]}{name[c[4]]}-{name[c[5]]}p{c[6]}-" + "_".join(f"{b}+{a}" for a, b in zip(c[7], c[8]))


@pytest.mark.parametrize("exact_max", [True, False], ids=["max_new", "any"])
@pytest.mark.parametrize("H,H_kv,d,s,dtype,kind,page,lens,starts", PAGED, ids=[_pid(c) for c in PAGED])
def test_paged_matches_plain(H, H_kv, d, s, dtype, kind, page, lens, starts, exact_max):
    ends = [a + b if a else 0 for a, b in zip(lens, starts)]
    plan = _plan(H, H_kv, max(a + b for a, b in zip(lens, starts)) + 11, d, s, dtype)
    g = _gen(sum(ends))
    pt, num = _table_of(ends, page)
    cache = _cache(num, H_kv, page, d, kind)
    K, V = _fill(cache, ends, pt, g, H_kv, d, dtype)
    T = sum(lens)
    q = _randn(g, T + 2, H, d, dtype=dtype)
    out = (torch.full((T + 2, H, d), 3.0, dtype=dtype, device="cuda:0"), torch.full((T + 2, H), 3.0, device="cuda:0"))
    O, R = plan.attend_paged(q, cache, pt, _cu(lens), torch.tensor(starts, dtype=torch.int32, device="cuda:0"),
                             max_new=max(lens) if exact_max else None, out=out)
    plan.check()
    assert (O[T:] == 3.0).all() and (R[T:] == 3.0).all()
    t = at = 0
    for n, (L, a) in enumerate(zip(lens, starts)):
        if L:
            want = plain.sequence(q[t:t + L].double(), K[at:at + a + L], V[at:at + a + L], plan.table_host, a)
            plain.check(O[t:t + L], R[t:t + L], want, dtype, f"sequence {n}")
        t += L
        at += ends[n]


@pytest.mark.parametrize("sigma", [0.3, 5000.0])
@pytest.mark.parametrize("kind,d,dtype", [(E4M3, 128, BF16), (BF16, 64, BF16), (F32, 64, F32)])
def test_paged_extreme_block_sizes(kind, d, dtype, sigma):
    lens, starts, page = [1, 1, 200, 3], [1500, 0, 900, 1300], 64
    ends = [a + b for a, b in zip(lens, starts)]
    plan, g = _plan(4, 2, 2000, d, 20, dtype, sigma=[sigma, 1.1 * sigma, 1.2 * sigma, 2 * sigma]), _gen(33)
    pt, num = _table_of(ends, page)
    cache = _cache(num, 2, page, d, kind)
    K, V = _fill(cache, ends, pt, g, 2, d, dtype)
    q, st = _randn(g, sum(lens), 4, d, dtype=dtype), torch.tensor(starts, dtype=torch.int32, device="cuda:0")
    O, R = plan.attend_paged(q, cache, pt, _cu(lens), st)
    plan.check()
    t = at = 0
    for n, (L, a) in enumerate(zip(lens, starts)):
        want = plain.sequence(q[t:t + L].double(), K[at:at + a + L], V[at:at + a + L], plan.table_host, a)
        plain.check(O[t:t + L], R[t:t + L], want, dtype, f"sequence {n}")
        t, at = t + L, at + ends[n]


def test_paged_sequences_may_share_pages():
    """Two sequences with a common prefix in the same pages, each with its own last page."""
    H, H_kv, d, page = 4, 2, 128, 64
    plan, g = _plan(H, H_kv, 400, d, 20, BF16), _gen(34)
    cache = _cache(8, H_kv, page, d, E4M3)
    pt = torch.tensor([[3, 1, 6, 0], [3, 1, 2, 0]], dtype=torch.int32, device="cuda:0")
    prefix, zero = _randn(g, 2, 128, H_kv, d), torch.zeros(1, dtype=torch.int32, device="cuda:0")
    cache.append(prefix[0], prefix[1], pt[:1].contiguous(), _cu([128]), zero)
    own = _randn(g, 2, 20, H_kv, d)
    start = torch.tensor([128, 128], dtype=torch.int32, device="cuda:0")
    cache.append(own[0], own[1], pt, _cu([10, 10]), start)
    q = _randn(g, 20, H, d)
    O, R = plan.attend_paged(q, cache, pt, _cu([10, 10]), start, max_new=10)
    plan.check()
    K, V = cache.read(pt, _cu([138, 138]), torch.zeros(2, dtype=torch.int32, device="cuda:0"), 276, dtype=F32)
    cache.check()
    assert torch.equal(K[:128], K[138:266])
    for n in range(2):
        want = plain.sequence(q[10 * n:10 * n + 10].double(), K[138 * n:138 * n + 138].double(), V[138 * n:138 * n + 138].double(),
                              plan.table_host, 128)
        plain.check(O[10 * n:10 * n + 10], R[10 * n:10 * n + 10], want, BF16)


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("kind,d,dtype", [(E4M3, 128, BF16), (BF16, 128, BF16), (E4M3, 64, BF16), (F32, 64, F32)])
def test_prompt_then_chunk_then_tokens(kind, d, dtype):
    """A server's run: prompts packed, into the cache, a chunk more of each, then tokens one by one; every step's rows against
    the whole sequence at once. The prompt sees its K and V as given, later steps as the cache holds them."""
    H, H_kv, page, prompts, chunk, steps = 4, 2, 32, [150, 1, 64], 70, 3
    S = len(prompts)
    plan, g = _plan(H, H_kv, 400, d, 20, dtype), _gen(40)
    ends = [p + chunk + steps for p in prompts]
    pt, num = _table_of(ends, page)
    cache = _cache(num, H_kv, page, d, kind)
    q, k, v = _randn(g, sum(prompts), H, d, dtype=dtype), *_randn(g, 2, sum(prompts), H_kv, d, dtype=dtype)
    start = torch.zeros(S, dtype=torch.int32, device="cuda:0")
    O, R = plan.attend_packed(q, k, v, _cu(prompts))
    cache.append(k, v, pt, _cu(prompts), start)
    _check_packed(plan, O, R, q, k, v, prompts)
    at = list(prompts)
    for n in [chunk] + [1] * steps:
        lens = [n] * S
        q, k, v = _randn(g, n * S, H, d, dtype=dtype), *_randn(g, 2, n * S, H_kv, d, dtype=dtype)
        start = torch.tensor(at, dtype=torch.int32, device="cuda:0")
        cache.append(k, v, pt, _cu(lens), start)
        O, R = plan.attend_paged(q, cache, pt, _cu(lens), start, max_new=n)
        at = [a + n for a in at]
        K, V = cache.read(pt, _cu(at), torch.zeros(S, dtype=torch.int32, device="cuda:0"), sum(at), dtype=F32 if cache.quantised else dtype)
        plan.check()
        cache.check()
        x = 0
        for s in range(S):
            want = plain.sequence(q[n * s:n * s + n].double(), K[x:x + at[s]].double(), V[x:x + at[s]].double(), plan.table_host, at[s] - n)
            plain.check(O[n * s:n * s + n], R[n * s:n * s + n], want, dtype, f"{n} tokens, sequence {s}")
            x += at[s]


def test_decoding_step_captured_and_replayed_on_another_stream():
    H, H_kv, d, page, S = 4, 2, 128, 64, 3
    plan, g = _plan(H, H_kv, 300, d, 20, BF16), _gen(41)
    pt, num = _table_of([300] * S, page)
    cache = _cache(num, H_kv, page, d, E4M3)
    _fill(cache, [200] * S, pt, g, H_kv, d, BF16)
    q, kv, start = _randn(g, S, H, d), _randn(g, 2, S, H_kv, d), torch.tensor([200] * S, dtype=torch.int32, device="cuda:0")
    cu = _cu([1] * S)
    packed = _randn(g, S, H, d), *_randn(g, 2, S, H_kv, d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cache.append(kv[0], kv[1], pt, cu, start)
        plan.attend_paged(q, cache, pt, cu, start, max_new=1)
        plan.attend_packed(*packed, cu)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs of the same step
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            cache.append(kv[0], kv[1], pt, cu, start)
            out = plan.attend_paged(q, cache, pt, cu, start, max_new=1)
            chunk = plan.attend_paged(q, cache, pt, cu, start)
            whole = plan.attend_packed(*packed, cu)
        graphs.append((graph, out, chunk, whole))
    for step in range(3):
        q.copy_(_randn(g, S, H, d))
        kv.copy_(_randn(g, 2, S, H_kv, d))
        start.fill_(200 + step)  # every position before it has been written
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for (graph, *_), stx in zip(graphs, streams):
            with torch.cuda.stream(stx):
                graph.replay()
        torch.cuda.synchronize()
        want = plan.attend_paged(q, cache, pt, cu, start, max_new=1)
        wchunk = plan.attend_paged(q, cache, pt, cu, start)
        wpack = plan.attend_packed(*packed, cu)
        for _, out, chunk, whole in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
            assert all(torch.equal(a, b) for a, b in zip(chunk, wchunk))
            assert all(torch.equal(a, b) for a, b in zip(whole, wpack))
    plan.check()
    cache.check()


def test_calls_on_a_stream_of_their_own():
    H, H_kv, d = 4, 2, 128
    plan, g = _plan(H, H_kv, 300, d, 20, BF16), _gen(42)
    q, k, v = _randn(g, 300, H, d), _randn(g, 300, H_kv, d), _randn(g, 300, H_kv, d)
    cu = _cu([100, 200])
    want = plan.attend_packed(q, k, v, cu)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = plan.attend_packed(q, k, v, cu, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_the_same_call_twice_gives_the_same_bits():
    H, H_kv, d, lens, starts = 8, 2, 128, [1, 300, 5, 1], [1800, 900, 64, 5]
    ends = [a + b for a, b in zip(lens, starts)]
    plan, g = _plan(H, H_kv, 2000, d, 20, BF16), _gen(43)
    pt, num = _table_of(ends, 64)
    cache = _cache(num, H_kv, 64, d, E4M3)
    _fill(cache, ends, pt, g, H_kv, d, BF16)
    q, st = _randn(g, sum(lens), H, d), torch.tensor(starts, dtype=torch.int32, device="cuda:0")
    first = plan.attend_paged(q, cache, pt, _cu(lens), st)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, plan.attend_paged(q, cache, pt, _cu(lens), st)))


# ---------------------------------------------------------------- empty and malformed calls


def test_empty_calls():
    plan, cache = _plan(2, 1, 100, 64, 8, BF16), _cache(2, 1, 16, 64, E4M3)
    none, one = torch.empty((0, 2, 64), dtype=BF16, device="cuda:0"), torch.empty((0, 1, 64), dtype=BF16, device="cuda:0")
    cu0 = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    pt = torch.zeros((1, 1), dtype=torch.int32, device="cuda:0")
    st = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    O, R = plan.attend_packed(none, one, one, cu0)
    assert O.shape == (0, 2, 64) and R.shape == (0, 2)
    plan.attend_packed(none, one, one, _cu([0, 0]))
    cache.append(one, one, pt, _cu([0]), st)
    K, V = cache.read(pt, _cu([0]), st, 0)
    assert K.shape == (0, 1, 64)
    plan.attend_paged(none, cache, pt, _cu([0]), st)
    # sequences without tokens beside a tensor with some
    x = torch.ones((3, 2, 64), dtype=BF16, device="cuda:0")
    O = torch.full((3, 2, 64), 2.0, dtype=BF16, device="cuda:0")
    R = torch.full((3, 2), 2.0, device="cuda:0")
    plan.attend_packed(x, x[:, :1], x[:, :1], _cu([0, 0]), out=(O, R))
    plan.attend_paged(x, cache, pt, _cu([0]), st, out=(O, R))
    plan.check()
    cache.check()
    assert (O == 2.0).all() and (R == 2.0).all()


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 64)])
def test_malformed_sequences_are_reported_and_skipped(dtype, d):
    plan, g = _plan(2, 1, 100, d, 8, dtype), _gen(50)
    cache = _cache(8, 1, 64, d, dtype)
    q, k, v = _randn(g, 150, 2, d, dtype=dtype), *_randn(g, 2, 150, 1, d, dtype=dtype)
    pt = torch.arange(8, dtype=torch.int32, device="cuda:0").view(2, 4)
    zero = torch.zeros(2, dtype=torch.int32, device="cuda:0")
    for cu in ([0, 50, 40], [0, 101, 150], [-3, 20, 90], [0, 10, 151]):
        cut = torch.tensor(cu, dtype=torch.int32, device="cuda:0")
        O = torch.full((150, 2, d), 2.0, dtype=dtype, device="cuda:0")
        R = torch.full((150, 2), 2.0, device="cuda:0")
        plan.attend_packed(q, k, v, cut, out=(O, R))
        assert plan.device_errors() == ["SEQUENCE"], cu
        plan.reset_errors()
        for n, (a, b) in enumerate(zip(cu, cu[1:])):
            good = 0 <= a <= b <= 150 and b - a <= 100
            if not good and 0 <= a < b <= 150:
                assert (O[a:b][~torch.isin(torch.arange(a, b), torch.arange(max(0, cu[1 - n]), max(0, cu[2 - n])))] == 2.0).all()
        plan.attend_paged(q, cache, pt, cut, zero, out=(O, R))
        assert "SEQUENCE" in plan.device_errors(), cu
        plan.reset_errors()
    cache.append(k, v, pt, torch.tensor([0, 50, 40], dtype=torch.int32, device="cuda:0"), zero)
    assert cache.device_errors() == ["SEQUENCE"]
    cache.reset_errors()
    # more new tokens than max_new, and a position behind max_len
    plan.attend_paged(q[:60], cache, pt, _cu([50, 10]), zero, max_new=20)
    assert plan.device_errors() == ["SEQUENCE"]
    plan.reset_errors()
    plan.attend_paged(q[:2], cache, pt, _cu([1, 1]), torch.tensor([100, 5], dtype=torch.int32, device="cuda:0"), max_new=1)
    assert "SEQUENCE" in plan.device_errors()


@pytest.mark.parametrize("kind,d,dtype", [(E4M3, 128, BF16), (BF16, 64, BF16), (F32, 64, F32)])
def test_pages_outside_the_pool_are_reported(kind, d, dtype):
    plan, g = _plan(2, 1, 400, d, 8, dtype, sigma=[500.0, 500.0]), _gen(51)
    cache = _cache(4, 1, 64, d, kind)
    cache.k_pages.view(torch.uint8).zero_()
    cache.v_pages.view(torch.uint8).zero_()
    kv = _randn(g, 2, 100, 1, d, dtype=dtype)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    for row in ([0, 4], [0, -1], [0]):  # behind the pool, before it, and a table too narrow
        pt = torch.tensor([row], dtype=torch.int32, device="cuda:0")
        cache.append(kv[0], kv[1], pt, _cu([100]), zero)
        assert cache.device_errors() == ["PAGE"], row
        cache.reset_errors()
        cache.read(pt, _cu([100]), zero, 100)
        assert cache.device_errors() == ["PAGE"], row
        cache.reset_errors()
        for lens, start in (([100], 0), ([1], 99)):
            plan.attend_paged(_randn(g, lens[0], 2, d, dtype=dtype), cache, pt, _cu(lens),
                              torch.tensor([start], dtype=torch.int32, device="cuda:0"), max_new=lens[0])
            assert plan.device_errors() == ["PAGE"], (row, lens)
            plan.reset_errors()


def test_refusals_of_the_python_layer():
    plan, cache = _plan(4, 2, 100, 128, 8, BF16), _cache(2, 2, 16, 128, E4M3)
    q, k = torch.zeros((8, 4, 128), dtype=BF16, device="cuda:0"), torch.zeros((8, 2, 128), dtype=BF16, device="cuda:0")
    cu, st, pt = _cu([8]), torch.zeros(1, dtype=torch.int32, device="cuda:0"), torch.zeros((1, 1), dtype=torch.int32, device="cuda:0")
    for args in ((q[:, :3], k, k, cu), (q, k[:7], k, cu), (q.float(), k, k, cu), (q, k, k.cpu(), cu), (q, k, k, cu.long()), (q, k, k, cu.cpu()),
                 (q, k[:, :1].expand(8, 2, 128), k, cu), (q.transpose(1, 2).contiguous().transpose(1, 2), k, k, cu),
                 (torch.zeros((8, 4, 130), dtype=BF16, device="cuda:0")[..., 1:129], k, k, cu)):
        with pytest.raises(ValueError):
            plan.attend_packed(*args)
    with pytest.raises(ValueError):
        plan.attend_packed(q, k, k, cu, out=(q.float(), torch.zeros((8, 4), device="cuda:0")))
    for args in ((q, cache, pt[0], cu, st), (q, cache, pt, cu, st.long()), (q, cache, pt, _cu([4, 4]), st),
                 (q, _cache(2, 1, 16, 128, E4M3), pt, cu, st), (q, _cache(2, 2, 16, 64, E4M3), pt, cu, st), (q, _cache(2, 2, 16, 128, F32), pt, cu, st)):
        with pytest.raises(ValueError):
            plan.attend_paged(*args)
    with pytest.raises(ValueError):
        plan.attend_paged(q, cache, pt, cu, st, max_new=0)
    with pytest.raises(ValueError):
        cache.append(k, k[:, :1], pt, cu, st)
    with pytest.raises(ValueError):
        cache.append(k.half(), k.half(), pt, cu, st)
    with pytest.raises(ValueError):
        cache.read(pt, cu, st, 8, dtype=torch.float16)
    with pytest.raises(ValueError):
        _cache(2, 2, 16, 128, BF16).append(k.float(), k.float(), pt, cu, st)
    plan.check()


# ---------------------------------------------------------------- at the edges


@pytest.mark.parametrize("d,dtype", [(128, BF16), (64, BF16), (64, F32)])
def test_a_rows_only_key_gives_its_value_exactly(d, dtype):
    """One key: O is its V, whatever the score (the weight and the sum are rounded alike), and row_sum the score."""
    H, H_kv, S = 6, 3, 40
    plan, g = _plan(H, H_kv, 64, d, 20, dtype), _gen(60)
    q, k, v = _randn(g, S, H, d, dtype=dtype), *_randn(g, 2, S, H_kv, d, dtype=dtype)
    want = v.repeat_interleave(2, 1)
    # one product p V, one quotient (p V) (1 / p): 2^-24 each and the reciprocal's 2^-23, far inside half a step of bf16
    near = 2.0 ** -22 if dtype == F32 else 0.0
    cu, zero = _cu([1] * S), torch.zeros(S, dtype=torch.int32, device="cuda:0")
    O, R = plan.attend_packed(q, k, v, cu)
    score = (q.double() * k.double().repeat_interleave(2, 1)).sum(-1) / d ** 0.5
    e = (d + 4) * 2.0 ** -23 * (q.double() * k.double().repeat_interleave(2, 1)).abs().sum(-1) / d ** 0.5
    assert ((O.double() - want.double()).abs() <= near * want.double().abs()).all()
    assert ((R.double() - score).abs() <= e + 2.0 ** -20 + 2.0 ** -22 * score.abs()).all()
    pt = torch.arange(S, dtype=torch.int32, device="cuda:0").view(S, 1)
    cache = _cache(S, H_kv, 16, d, dtype)
    cache.append(k, v, pt, cu, zero)
    for most in (1, None):
        O, R = plan.attend_paged(q, cache, pt, cu, zero, max_new=most)
        assert ((O.double() - want.double()).abs() <= near * want.double().abs()).all()
        assert ((R.double() - score).abs() <= e + 2.0 ** -20 + 2.0 ** -22 * score.abs()).all()
    plan.check()
    cache.check()


@pytest.mark.parametrize("H,H_kv,lens,starts", [
    (72, 72, [1, 2], [100, 0]),            # more KV heads than the rows kernel splits one by one
    (80, 80, [40, 1, 3], [7, 130, 64]),
    (24, 2, [1, 5], [300, 64]),            # twelve query heads to a KV head: two blocks of them
    (24, 2, [70, 1, 2], [30, 200, 5]),
    (264, 8, [150, 1], [0, 90]),           # more heads than the tile kernel sorts
])
def test_paged_many_heads(H, H_kv, lens, starts):
    d, page = 64, 32
    ends = [a + b for a, b in zip(lens, starts)]
    plan, g = _plan(H, H_kv, max(ends) + 3, d, 12, BF16), _gen(61)
    pt, num = _table_of(ends, page)
    cache = _cache(num, H_kv, page, d, E4M3)
    K, V = _fill(cache, ends, pt, g, H_kv, d, BF16)
    q, st = _randn(g, sum(lens), H, d), torch.tensor(starts, dtype=torch.int32, device="cuda:0")
    O, R = plan.attend_paged(q, cache, pt, _cu(lens), st, max_new=max(lens))
    plan.check()
    t = at = 0
    for n, (L, a) in enumerate(zip(lens, starts)):
        want = plain.sequence(q[t:t + L].double(), K[at:at + a + L], V[at:at + a + L], plan.table_host, a)
        plain.check(O[t:t + L], R[t:t + L], want, BF16, f"sequence {n}")
        t, at = t + L, at + ends[n]
    T = sum(ends)
    q = _randn(g, T, H, d)
    O, R = plan.attend_packed(q, K.to(BF16), V.to(BF16), _cu(ends))
    plan.check()
    _check_packed(plan, O, R, q, K.to(BF16), V.to(BF16), ends)


@pytest.mark.parametrize("kind,d,dtype", [(E4M3, 128, BF16), (F32, 64, F32)])
def test_thousands_of_sequences(kind, d, dtype):
    # more than 32 x 32: three steps of the search for a tile's sequence; empty ones in between
    H, H_kv, page, S = 4, 2, 16, 2500
    g, rng = _gen(69), np.random.default_rng(2)
    lens = [int(x) for x in rng.choice([0, 1, 1, 2, 5], S)]
    starts = [int(x) for x in rng.integers(0, 60, S)]
    ends = [a + b if a else 0 for a, b in zip(lens, starts)]
    plan = _plan(H, H_kv, 80, d, 20, dtype)
    pt, num = _table_of(ends, page)
    cache = _cache(num, H_kv, page, d, kind)
    K, V = _fill(cache, ends, pt, g, H_kv, d, dtype)
    q, st = _randn(g, sum(lens), H, d, dtype=dtype), torch.tensor(starts, dtype=torch.int32, device="cuda:0")
    kp, vp = K.to(dtype), V.to(dtype)
    qp = _randn(g, sum(ends), H, d, dtype=dtype)
    OP, RP = plan.attend_packed(qp, kp, vp, _cu(ends))
    for most in (5, None):
        O, R = plan.attend_paged(q, cache, pt, _cu(lens), st, max_new=most)
        plan.check()
        t, at = np.concatenate([[0], np.cumsum(lens)]), np.concatenate([[0], np.cumsum(ends)])
        for n in list(range(0, S, 97)) + [S - 2, S - 1]:
            if not lens[n]:
                continue
            a, b = slice(t[n], t[n + 1]), slice(at[n], at[n + 1])
            plain.check(O[a], R[a], plain.sequence(q[a].double(), K[b], V[b], plan.table_host, starts[n]), dtype, f"sequence {n}")
            plain.check(OP[b], RP[b], plain.sequence(qp[b].double(), kp[b].double(), vp[b].double(), plan.table_host, 0), dtype, f"prompt {n}")


@pytest.mark.parametrize("kind", [E4M3, BF16])
def test_a_chunk_among_many_single_tokens(kind):
    # many short sequences beside the tile kernel's: the rows kernel's, of up to 8 rows each
    H, H_kv, d, page, lens = 16, 8, 64, 32, [1] * 24 + [70, 0, 4, 5] + [2] * 22
    g, rng = _gen(68), np.random.default_rng(1)
    starts = [int(x) for x in rng.integers(0, 150, len(lens))]
    ends = [a + b for a, b in zip(lens, starts)]
    plan = _plan(H, H_kv, max(ends), d, 20, BF16)
    pt, num = _table_of(ends, page)
    cache = _cache(num, H_kv, page, d, kind)
    K, V = _fill(cache, ends, pt, g, H_kv, d, BF16)
    q, st = _randn(g, sum(lens), H, d), torch.tensor(starts, dtype=torch.int32, device="cuda:0")
    for most in (70, None):
        O, R = plan.attend_paged(q, cache, pt, _cu(lens), st, max_new=most)
        plan.check()
        t = at = 0
        for n, (L, a) in enumerate(zip(lens, starts)):
            if L:
                want = plain.sequence(q[t:t + L].double(), K[at:at + a + L], V[at:at + a + L], plan.table_host, a)
                plain.check(O[t:t + L], R[t:t + L], want, BF16, f"sequence {n}")
            t, at = t + L, at + ends[n]


@pytest.mark.parametrize("lens", [[1, 4, 5, 16, 17], [16, 1, 16], [3, 17, 2, 4]])
def test_sequences_on_either_side_of_the_kernels_limits(lens):
    # 8 rows, here 4 tokens, of a block; 16 tokens of the rows kernel's longest call
    H, H_kv, d, page, starts = 4, 2, 128, 16, [90, 0, 33, 15, 64][:len(lens)]
    ends = [a + b for a, b in zip(lens, starts)]
    plan, g = _plan(H, H_kv, 200, d, 20, BF16), _gen(62)
    pt, num = _table_of(ends, page)
    cache = _cache(num, H_kv, page, d, E4M3)
    K, V = _fill(cache, ends, pt, g, H_kv, d, BF16)
    q, st = _randn(g, sum(lens), H, d), torch.tensor(starts, dtype=torch.int32, device="cuda:0")
    for most in (max(lens), None):
        O, R = plan.attend_paged(q, cache, pt, _cu(lens), st, max_new=most)
        plan.check()
        t = at = 0
        for n, (L, a) in enumerate(zip(lens, starts)):
            want = plain.sequence(q[t:t + L].double(), K[at:at + a + L], V[at:at + a + L], plan.table_host, a)
            plain.check(O[t:t + L], R[t:t + L], want, BF16, f"sequence {n}")
            t, at = t + L, at + ends[n]


@pytest.mark.parametrize("most", [8, 9, 16])
@pytest.mark.parametrize("S", [8, 20])
@pytest.mark.parametrize("kind", [E4M3, BF16])
def test_chunks_of_several_tokens_in_large_and_small_calls(kind, S, most):
    H, H_kv, d, page = 2, 1, 64, 32
    g, rng = _gen(67), np.random.default_rng(most)
    lens = [most] + [int(x) for x in rng.integers(1, most + 1, S - 1)]
    starts = [int(x) for x in rng.integers(0, 150, S)]
    ends = [a + b for a, b in zip(lens, starts)]
    plan = _plan(H, H_kv, max(ends), d, 20, BF16)
    pt, num = _table_of(ends, page)
    cache = _cache(num, H_kv, page, d, kind)
    K, V = _fill(cache, ends, pt, g, H_kv, d, BF16)
    q, st = _randn(g, sum(lens), H, d), torch.tensor(starts, dtype=torch.int32, device="cuda:0")
    O, R = plan.attend_paged(q, cache, pt, _cu(lens), st, max_new=most)
    plan.check()
    t = at = 0
    for n, (L, a) in enumerate(zip(lens, starts)):
        want = plain.sequence(q[t:t + L].double(), K[at:at + a + L], V[at:at + a + L], plan.table_host, a)
        plain.check(O[t:t + L], R[t:t + L], want, BF16, f"sequence {n}")
        t, at = t + L, at + ends[n]


@pytest.mark.parametrize("kind", [E4M3, BF16])
def test_a_pool_past_32_bit_offsets(kind):
    """Pages whose first element lies past 2^32 elements of the pool."""
    from alibi_positional_lsh_b200 import PagedCache
    H, H_kv, d, page = 4, 1, 128, 256
    num = (1 << 32) // (page * H_kv * d) + 4
    cache = PagedCache.empty(num, H_kv, page, d, kind, "cuda:0")
    pt = torch.tensor([[num - 1, num - 3], [num - 2, num - 4]], dtype=torch.int32, device="cuda:0")
    plan, g = _plan(H, H_kv, 512, d, 20, BF16), _gen(63)
    ends, zero = [400, 290], torch.zeros(2, dtype=torch.int32, device="cuda:0")
    k, v = _randn(g, 2, 690, H_kv, d)
    cache.append(k, v, pt, _cu(ends), zero)
    K, V = cache.read(pt, _cu(ends), zero, 690)
    cache.check()
    if kind == BF16:
        assert torch.equal(K, k) and torch.equal(V, v)
    else:  # half a step of e4m3 relative to the row's scale: 2^-4 of a value, 2^-10 of 2^e below its normal numbers
        assert ((K.double() - k.double()).abs() <= 2.0 ** -4 * k.double().abs() + 2.0 ** -10 * k.double().abs().amax(-1, keepdim=True) / 224).all()
    for n in (1, 30):
        q, st = _randn(g, 2 * n, H, d), torch.tensor([400 - n, 290 - n], dtype=torch.int32, device="cuda:0")
        O, R = plan.attend_paged(q, cache, pt, _cu([n, n]), st, max_new=n)
        plan.check()
        for s, (a, b) in enumerate(((0, 400), (400, 690))):
            want = plain.sequence(q[n * s:n * s + n].double(), K[a:b].double(), V[a:b].double(), plan.table_host, b - a - n)
            plain.check(O[n * s:n * s + n], R[n * s:n * s + n], want, BF16, f"{n} tokens, sequence {s}")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite_spoils_its_own_row_only(bad):
    H, H_kv, d, page = 4, 2, 128, 64
    plan, g = _plan(H, H_kv, 300, d, 20, BF16), _gen(64)
    pt, num = _table_of([250], page)
    cache = _cache(num, H_kv, page, d, E4M3)
    K, V = _fill(cache, [250], pt, g, H_kv, d, BF16)
    for n in (3, 100, 250):
        q, st = _randn(g, n, H, d), torch.tensor([250 - n], dtype=torch.int32, device="cuda:0")
        call = (lambda: plan.attend_packed(q, K.to(BF16), V.to(BF16), _cu([n]))) if n == 250 else \
               (lambda: plan.attend_paged(q, cache, pt, _cu([n]), st, max_new=n))
        O, R = call()
        q[1, 2, 5] = bad
        O2, R2 = call()
        plan.check()
        keep = torch.ones((n, H), dtype=torch.bool, device="cuda:0")
        keep[1, 2] = False
        assert torch.equal(O[keep], O2[keep]) and torch.equal(R[keep], R2[keep]), n
        assert not torch.isfinite(O2[1, 2]).all()


def test_near_counts_against_the_bins():
    H, n = 3, 200
    for s in (1, 20, 64):
        plan = _plan(H, 1, n, 64, s, BF16, sigma=[1.0, 9.0, 200.0])
        ids = oracle.bin_ids(plan.table_host, n)
        near = plan.near.cpu().numpy()
        for h in range(H):
            c = (ids[h][:, :, None] == ids[h][:, None, :]).sum(0)  # [n][n], over the hashes
            for p in range(n):
                row = np.zeros(64, dtype=np.int64)
                j = np.arange(p // 64 * 64, p + 1)
                row[j % 64] = c[p, j]
                assert (near[h, p] == row).all(), (s, h, p)


def test_the_plain_entry_points_give_the_same_bits():
    import alibi_positional_lsh_b200 as m
    H, H_kv, d, s, page, lens = 4, 2, 128, 20, 64, [40, 1, 30]
    plan, g, T = _plan(H, H_kv, 100, d, s, BF16), _gen(65), 71
    q, k, v = _randn(g, T, H, d), *_randn(g, 2, T, H_kv, d)
    cu, zero = _cu(lens), torch.zeros(3, dtype=torch.int32, device="cuda:0")
    err = torch.zeros(4, dtype=torch.int32, device="cuda:0")
    near = torch.empty_like(plan.near)
    m.plsh_near_counts(plan.bmask, H, s, 100, near)
    assert torch.equal(near, plan.near)
    O, R = torch.empty_like(q), torch.empty((T, H), device="cuda:0")
    m.plsh_packed_fwd(q, k, v, m.PLSH_BF16, cu, H, H_kv, d, s, 100, plan.spans, plan.bmask, near, O, R, err)
    assert all(torch.equal(a, b) for a, b in zip((O, R), plan.attend_packed(q, k, v, cu)))
    pt, num = _table_of(lens, page)
    a, b = _cache(num, H_kv, page, d, E4M3), _cache(num, H_kv, page, d, E4M3)
    a.append(k, v, pt, cu, zero)
    m.plsh_cache_append(k, v, m.PLSH_BF16, cu, zero, H_kv, d, b.k_pages, b.v_pages, b.k_exp, b.v_exp, pt, err)
    for x, y in zip((a.k_pages, a.v_pages, a.k_exp, a.v_exp), (b.k_pages, b.v_pages, b.k_exp, b.v_exp)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    K, V = torch.empty_like(k), torch.empty_like(v)
    m.plsh_cache_read(b.k_pages, b.v_pages, b.k_exp, b.v_exp, pt, cu, zero, H_kv, d, m.PLSH_BF16, K, V, err)
    assert all(torch.equal(x, y) for x, y in zip((K, V), a.read(pt, cu, zero, T)))
    scratch = torch.empty(m.plsh_paged_scratch_bytes(T, 3, T, H_kv, d, plan.max_window), dtype=torch.uint8, device="cuda:0")
    m.plsh_paged_fwd(q, m.PLSH_BF16, cu, zero, T, H, H_kv, d, b.k_pages, b.v_pages, b.k_exp, b.v_exp, pt, s, 100, plan.table_dev,
                     plan.spans, plan.bmask, near, plan.windows_host, scratch, O, R, err)
    assert all(torch.equal(x, y) for x, y in zip((O, R), plan.attend_paged(q, a, pt, cu, zero)))
    assert int(err.abs().max()) == 0


@pytest.mark.parametrize("paged", [False, True])
def test_a_bounded_wait_runs_out_and_the_next_call_is_correct(paged):
    """The tile kernel's issuer of tensor-core products told to issue none: every wait for scores runs out after the limit, the
    launch reports it and returns, and the next call on the same context is right."""
    from alibi_positional_lsh_b200 import plsh_set_wait_limit_ns, plsh_test_withhold_mma
    H, H_kv, d, page, lens = 2, 1, 128, 64, [300, 90]
    plan, g = _plan(H, H_kv, 300, d, 12, BF16), _gen(66)
    q, k, v = _randn(g, 390, H, d), *_randn(g, 2, 390, H_kv, d)
    cu, zero = _cu(lens), torch.zeros(2, dtype=torch.int32, device="cuda:0")
    pt, num = _table_of(lens, page)
    cache = _cache(num, H_kv, page, d, BF16)
    cache.append(k, v, pt, cu, zero)
    call = (lambda: plan.attend_paged(q, cache, pt, cu, zero)) if paged else (lambda: plan.attend_packed(q, k, v, cu))
    call()
    plan.check()
    plsh_set_wait_limit_ns(1_000_000)
    plsh_test_withhold_mma(True)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        plsh_test_withhold_mma(False)
        plsh_set_wait_limit_ns(0)
    assert "TIMEOUT" in plan.device_errors()
    plan.reset_errors()
    O, R = call()
    plan.check()
    _check_packed(plan, O, R, q, k, v, lens)

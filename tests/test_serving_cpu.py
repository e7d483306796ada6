"""The serving entry points without a GPU: the host-side checks refuse bad arguments before any device work, and the
plain implementation that the GPU tests compare with agrees with the oracle."""
import ctypes
import struct

import numpy as np
import pytest
import torch

import oracle
from tests import serving_plain as plain

FAKE = ctypes.c_void_p(1 << 20)  # never dereferenced: the checks fail first
NULL = None


@pytest.fixture(scope="module")
def plsh():
    import alibi_positional_lsh_b200 as m
    return m


def _packed(Q=FAKE, qt=512, qh=128, kt=256, dtype=0, T=10, S=2, cu=FAKE, H=4, H_kv=2, d=128, s=20, max_len=100, spans=FAKE, near=FAKE, O=FAKE):
    return (Q, qt, qh, FAKE, kt, 128, FAKE, 256, 128, dtype, T, S, cu, H, H_kv, d, s, max_len, spans, FAKE, near, O, FAKE, FAKE, NULL)


def _append(K=FAKE, dtype=0, T=10, S=2, start=FAKE, d=128, kp=FAKE, ke=FAKE, ve=FAKE, width=3, pages=8, page=64):
    return (K, 256, 128, FAKE, 256, 128, dtype, T, S, FAKE, start, 2, d, kp, FAKE, ke, ve, FAKE, width, pages, page, FAKE, NULL)


def _read(kp=FAKE, ke=FAKE, ve=FAKE, width=3, pages=8, page=64, T=10, start=FAKE, d=128, dtype=0, K=FAKE):
    return (kp, FAKE, ke, ve, FAKE, width, pages, page, T, 2, FAKE, start, 2, d, dtype, K, FAKE, FAKE, NULL)


def _paged(Q=FAKE, qt=512, dtype=0, T=10, S=2, start=FAKE, max_new=10, H=4, H_kv=2, d=128, ke=FAKE, ve=FAKE, page=64, s=20,
           max_len=100, table=FAKE, near=FAKE, window=50, windows=True, scratch=FAKE, nbytes=1 << 30, O=FAKE):
    return (Q, qt, 128, dtype, T, S, FAKE, start, max_new, H, H_kv, d, FAKE, FAKE, ke, ve, FAKE, 3, 8, page, s, max_len, table, FAKE, FAKE,
            near, (ctypes.c_int32 * 8)(window, 9, 9, 9, 9, 9, 9, 9) if windows else NULL, scratch, ctypes.c_size_t(nbytes), O, FAKE, FAKE, NULL)


ODD = ctypes.c_void_p((1 << 20) + 8)
REFUSED = [
    ("plsh_near_counts", lambda H=2, s=8, n=10, near=FAKE: (FAKE, H, s, n, near, NULL),
     [(dict(H=0), 1), (dict(s=65), 1), (dict(n=0), 1), (dict(near=NULL), 1), (dict(near=ODD), 1)]),
    ("plsh_packed_fwd", _packed, [(dict(Q=NULL), 1), (dict(Q=ODD), 1), (dict(qt=508), 1), (dict(qh=64), 1), (dict(kt=64), 1), (dict(dtype=7), 2),
                                  (dict(T=0), 1), (dict(S=0), 1), (dict(cu=NULL), 1), (dict(H_kv=3), 1), (dict(H=0), 1), (dict(d=96), 2),
                                  (dict(s=0), 1), (dict(s=65), 1), (dict(max_len=0), 1), (dict(spans=NULL), 1), (dict(near=NULL), 1), (dict(near=ODD), 1), (dict(O=ODD), 1),
                                  (dict(T=1 << 30, qt=1 << 20), 3), (dict(S=1 << 21), 3)]),
    ("plsh_cache_append", _append, [(dict(K=NULL), 1), (dict(dtype=2), 2), (dict(T=0), 1), (dict(S=0), 1), (dict(start=NULL), 1), (dict(d=32), 2),
                                    (dict(kp=NULL), 1), (dict(ke=NULL), 1), (dict(ve=NULL), 1), (dict(width=0), 1), (dict(pages=0), 1),
                                    (dict(page=48), 2), (dict(page=8), 2), (dict(page=512), 2)]),
    ("plsh_cache_read", _read, [(dict(kp=ODD), 1), (dict(ke=NULL), 1), (dict(width=0), 1), (dict(page=100), 2), (dict(T=0), 1),
                                (dict(start=NULL), 1), (dict(d=256), 2), (dict(dtype=5), 2), (dict(K=NULL), 1), (dict(K=ODD), 1)]),
    ("plsh_paged_fwd", _paged, [(dict(Q=NULL), 1), (dict(qt=100), 1), (dict(dtype=3), 2), (dict(T=0), 1), (dict(start=NULL), 1), (dict(max_new=0), 1),
                                (dict(H_kv=3), 1), (dict(d=80), 2), (dict(ve=NULL), 1), (dict(page=20), 2), (dict(s=99), 1), (dict(max_len=0), 1),
                                (dict(O=NULL), 1), (dict(table=NULL), 1), (dict(max_new=17, near=NULL), 1), (dict(window=101), 1), (dict(window=0), 1), (dict(windows=False), 1),
                                (dict(max_new=17, scratch=NULL), 1), (dict(max_new=17, nbytes=1000), 1)]),
]


@pytest.mark.parametrize("name,args,bad", REFUSED, ids=[r[0] for r in REFUSED])
def test_bad_arguments_are_refused_before_any_launch(plsh, name, args, bad):
    for change, code in bad:
        assert getattr(plsh._lib, name)(*args(**change)) == code, change
        assert plsh.plsh_last_error().startswith(name + ":")


@pytest.mark.parametrize("name,args,bad", REFUSED[1:], ids=[r[0] for r in REFUSED[1:]])
def test_the_same_refusals_through_an_array(plsh, name, args, bad):
    def call(values, cut=0):
        a = [ctypes.cast(x, ctypes.c_void_p).value if isinstance(x, ctypes.Array) else x.value if hasattr(x, "value") else x for x in values]
        raw = struct.pack(f"={len(a)}q", *[x or 0 for x in a])
        return getattr(plsh._lib, name + "_args")(raw, len(raw) - cut)
    for change, code in bad:
        values = args(**change)  # kept: the array holds addresses
        assert call(values) == code, change
    values = args(**bad[0][0])
    for cut in (8, -8):
        assert call(values, cut) == 1 and "bytes of arguments" in plsh.plsh_last_error()
    assert call(args(T=(1 << 32) + 10)) == 3 and "does not fit" in plsh.plsh_last_error()
    assert getattr(plsh._lib, name + "_args")(None, 8 * len(values)) == 1


def test_scratch_is_needed_by_tiles_of_e4m3_only(plsh):
    assert plsh.plsh_paged_scratch_bytes(100, 2, 16, 2, 128, 50) == 0
    assert plsh.plsh_paged_scratch_bytes(128, 8, 16, 2, 128, 50) == 0 and plsh.plsh_paged_scratch_bytes(4000, 500, 8, 2, 128, 50) == 0
    assert plsh.plsh_paged_scratch_bytes(129, 9, 16, 2, 128, 50) == 2 * (129 + 9 * 320) * 2 * 128 * 2
    assert plsh.plsh_paged_scratch_bytes(100, 2, 17, 2, 128, 50) == 2 * (100 + 2 * 320) * 2 * 128 * 2
    assert plsh.plsh_paged_scratch_bytes(0, 2, 17, 2, 128, 50) == 0


def test_plain_sequence_agrees_with_the_oracle():
    H, H_kv, n, d, s = 2, 1, 90, 64, 12
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((n, h, d), generator=g, dtype=torch.float64) for h in (H, H_kv, H_kv))
    table = oracle.draw_table(5, [3.0, 40.0], s)
    O, R, _, _ = plain.sequence(q, k, v, table, 0)
    tail, rt, _, _ = plain.sequence(q[60:], k, v, table, 60)
    for h in range(H):
        wO, wR = oracle.approx_attention(q[:, h].numpy(), k[:, 0].numpy(), v[:, 0].numpy(), oracle.bin_ids(table, n)[h], True)
        assert np.abs(O[:, h].numpy() - wO).max() <= 1e-12 and np.abs(R[:, h].numpy() - wR).max() <= 1e-12
    assert (tail - O[60:]).abs().max() <= 1e-13 and (rt - R[60:]).abs().max() <= 1e-13


def test_plain_quantiser_agrees_with_torch_and_keeps_its_definition():
    g = torch.Generator().manual_seed(2)
    x = torch.randn((40, 2, 64), generator=g) * torch.exp2(torch.randint(-20, 20, (40, 2, 1), generator=g).float())
    byte, exp = plain.quantise(x.double().numpy())
    top = x.abs().amax(-1).double().numpy()
    assert (top <= 448.0 * 2.0 ** exp).all() and (top > 448.0 * 2.0 ** (exp - 1.0)).all()
    scaled = x.double() * torch.exp2(-torch.tensor(exp).double())[..., None]
    assert np.array_equal(scaled.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy(), byte)
    assert np.array_equal(plain.values(byte, exp), scaled.float().to(torch.float8_e4m3fn).double().numpy() * (2.0 ** exp.astype(float))[..., None])


def test_what_the_calls_keep_addresses_of_cannot_be_exchanged(plsh):
    import copy
    from alibi_positional_lsh_b200.serving import _Kept

    class Kept(_Kept):
        def __init__(self):
            self.t, self.size = torch.arange(4), 4
            self._fix()

        def _keep(self):
            return {"_at": self.t.data_ptr()}

    x = Kept()
    for name in ("t", "size", "_at"):
        with pytest.raises(AttributeError):
            setattr(x, name, 1)
        with pytest.raises(AttributeError):
            delattr(x, name)
    x.note = "the caller's own"
    x.note = "which may change"
    x.other = 1
    del x.other
    for y in (copy.copy(x), copy.deepcopy(x)):
        assert y._at == y.t.data_ptr() and torch.equal(y.t, x.t) and y.note == x.note
        with pytest.raises(AttributeError):
            y.t = x.t
        y.note = "again"
    assert copy.deepcopy(x)._at != x._at
    assert issubclass(plsh.PagedCache, _Kept) and issubclass(plsh.PlshServing, _Kept)


def test_scratch_does_not_grow_with_all_sequences(plsh):
    # 64 and 1,024 sequences, one of them perhaps a chunk, with heads that reach back 100,000 tokens; one window is (100,000 + 256) rows up to whole 64
    one = 4 * 8 * 128 * 100288
    assert plsh.plsh_paged_scratch_bytes(600, 1, 512, 8, 128, 100_000) == 4 * 600 * 8 * 128 + one
    for S in (64, 1024):
        assert one <= plsh.plsh_paged_scratch_bytes(600, S, 512, 8, 128, 100_000) - 4 * 600 * 8 * 128 <= 2 << 30
    # a window that alone takes more than that
    assert plsh.plsh_paged_scratch_bytes(600, 64, 512, 64, 128, 100_000) == 8 * (4 * 600 * 8 * 128 + one)

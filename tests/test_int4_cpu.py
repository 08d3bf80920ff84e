"""Host-side checks of the 4-bit cache's and the q/k norm's entry points: sizes
and refusals, none of which reaches the device; and the oracle's own layout."""
import ctypes

import numpy as np
import pytest

import int4_util as I
import paged_kv_attention_photon_gb300 as P
import workloads as W

FAKE, FAKE2 = 0x10000, 0x20000   # aligned non-null addresses that are never read
OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    P.build()
    return P._load()


def _shape(**over):
    base = dict(num_seqs=4, num_q_heads=16, num_kv_heads=8, head_dim=128, block_size=16,
                num_blocks=100, max_blocks_per_seq=8, dtype=P.F16, partition_size=0)
    base.update(over)
    return P.PagedShape.make(**base)


BAD_SHAPES = [(dict(dtype=P.F32), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED),
              (dict(block_size=32), UNSUPPORTED), (dict(num_q_heads=40), UNSUPPORTED),
              (dict(num_q_heads=12), INVALID), (dict(num_seqs=-1), INVALID)]


def test_sizes(lib):
    assert P.photon_cache_int4_bytes(_shape()) == 100 * 8 * (8 * 128 + 64)
    assert P.photon_cache_int4_bytes(_shape(head_dim=64, num_blocks=3)) == 3 * 8 * 576
    assert P.photon_cache_int4_bytes(_shape(num_blocks=4_000_000)) == 4_000_000 * 8 * 1088
    assert P.photon_paged_decode_int4_workspace_size(_shape()) > 0
    assert P.photon_paged_decode_int4_workspace_size(_shape(num_seqs=0)) == 0
    for over, _ in BAD_SHAPES:
        assert P.photon_cache_int4_bytes(_shape(**over)) == 0
        assert P.photon_paged_decode_int4_workspace_size(_shape(**over)) == 0


def _write(lib, shape, k=FAKE, ks=0, v=FAKE, vs=0, slots=FAKE, n=3, kc=FAKE2, vc=FAKE2):
    return lib.photon_cache_write_int4(k, ks, v, vs, slots, n, kc, vc, ctypes.byref(shape), None)


def test_write_refusals(lib):
    for over, want in BAD_SHAPES:
        assert _write(lib, _shape(**over)) == want
    s = _shape()
    assert _write(lib, s, n=-1) == INVALID
    assert _write(lib, s, n=0, k=None) == OK
    assert _write(lib, s, ks=-1024) == INVALID
    assert _write(lib, s, ks=1016) == INVALID           # shorter than the row
    assert _write(lib, s, vs=1028) == MISALIGNED        # 2056 bytes
    for name in ("k", "v", "slots", "kc", "vc"):
        assert _write(lib, s, **{name: None}) == INVALID
        assert _write(lib, s, **{name: FAKE + 4}) == MISALIGNED


def test_gather_refusals(lib):
    def call(shape, *p):
        args = list(p) or [FAKE] * 6
        return lib.photon_paged_gather_int4(*args, ctypes.byref(shape), None)
    for over, want in BAD_SHAPES:
        assert call(_shape(**over)) == want
    assert call(_shape(num_seqs=0), *[None] * 6) == OK
    for i in range(6):
        for bad, want in ((None, INVALID), (FAKE + 8, MISALIGNED)):
            args = [FAKE] * 6
            args[i] = bad
            assert call(_shape(), *args) == want


def test_decode_refusals(lib):
    def call(shape, q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, cl=FAKE, scale=0.1, out=FAKE2, ws=FAKE2,
             n=1 << 40):
        return lib.photon_paged_decode_int4(q, kc, vc, bt, cl, scale, out, ws, n,
                                            ctypes.byref(shape), None)
    for over, want in BAD_SHAPES:
        assert call(_shape(**over)) == want
    s = _shape()
    need = P.photon_paged_decode_int4_workspace_size(s)
    assert call(s, n=need - 1) == WORKSPACE
    assert call(s, ws=None) == WORKSPACE
    assert call(s, ws=FAKE + 8) == MISALIGNED
    assert call(s, scale=float("nan")) == INVALID
    assert call(s, scale=float("inf")) == INVALID
    assert call(_shape(num_seqs=0), q=None) == OK
    for name in ("q", "kc", "vc", "bt", "cl", "out"):
        assert call(s, **{name: None}) == INVALID
        assert call(s, **{name: FAKE + 8}) == MISALIGNED
    assert call(_shape(num_seqs=65535, num_q_heads=60000, num_kv_heads=30000)) == UNSUPPORTED
    assert call(_shape(num_seqs=4096, max_blocks_per_seq=1 << 16)) == UNSUPPORTED
    assert call(_shape(num_blocks=1 << 28)) == UNSUPPORTED


def _qk(lib, shape, axes=None, q=FAKE, qs=0, k=FAKE, ks=0, qw=FAKE, kw=FAKE, eps=1e-6, pos=FAKE,
        cs=FAKE, max_pos=128, n=3, qo=FAKE2, qos=0, ko=FAKE2, kos=0):
    axes = P.RopeAxes.make([64]) if axes is None else axes
    return lib.photon_qk_norm_rope(q, qs, k, ks, qw, kw, eps, pos, cs, max_pos, ctypes.byref(axes),
                                   n, qo, qos, ko, kos, ctypes.byref(shape), None)


def test_qk_refusals(lib):
    for over, want in BAD_SHAPES[1:]:
        assert _qk(lib, _shape(**over)) == want
    s = _shape()
    assert _qk(lib, s, n=-1) == INVALID
    assert _qk(lib, s, n=0, q=None) == OK
    assert _qk(lib, s, max_pos=0) == INVALID
    for eps in (-1e-6, float("nan"), float("inf")):
        assert _qk(lib, s, eps=eps) == INVALID
    for name in ("q", "k", "pos", "cs", "qo", "ko"):
        assert _qk(lib, s, **{name: None}) == INVALID
    for name in ("q", "k", "qw", "kw", "cs", "qo", "ko"):
        assert _qk(lib, s, **{name: FAKE + 8}) == MISALIGNED
    assert _qk(lib, s, pos=FAKE + 2) == MISALIGNED
    for name, row in (("qs", 2048), ("ks", 1024), ("qos", 2048), ("kos", 1024)):
        assert _qk(lib, s, **{name: row - 8}) == INVALID
        assert _qk(lib, s, **{name: row + 4}) == MISALIGNED
        assert _qk(lib, s, **{name: -row}) == INVALID
    assert _qk(lib, _shape(dtype=P.F32), qs=2050) == MISALIGNED


def test_qk_axes_refusals(lib):
    s = _shape()
    for sections, dealt, want in [
            ([72], False, INVALID),                      # more pairs than the row has
            ([0], False, INVALID), ([32, -8], False, INVALID),
            ([20], False, UNSUPPORTED),                  # rotary_dim 40
            ([16, 16, 16, 16, 16], False, INVALID),      # five axes
            ([8, 28, 28], True, INVALID),                # axis 1 would reach past pair 63
    ]:
        assert _qk(lib, s, P.RopeAxes.make(sections, dealt)) == want, sections
    bad = P.RopeAxes.make([64])
    bad.interleaved = 2
    assert _qk(lib, s, bad) == INVALID
    bad = P.RopeAxes.make([64])
    bad.num_axes = 0
    assert _qk(lib, s, bad) == INVALID


def _prompt(lib, shape, q=FAKE, qs=0, k=FAKE, ks=0, v=FAKE, vs=0, start=FAKE, n=7, longest=7,
            scale=0.1, out=FAKE2, os=0):
    return lib.photon_prompt_attention(q, qs, k, ks, v, vs, start, n, longest, scale, out, os,
                                       ctypes.byref(shape), None)


def test_prompt_refusals(lib):
    for over, want in BAD_SHAPES:
        assert _prompt(lib, _shape(**over)) == want
    s = _shape()
    assert _prompt(lib, s, n=-1) == INVALID
    assert _prompt(lib, s, longest=-1) == INVALID
    for scale in (float("nan"), float("inf")):
        assert _prompt(lib, s, scale=scale) == INVALID
    assert _prompt(lib, s, n=0, q=None) == OK
    assert _prompt(lib, s, longest=0, q=None) == OK
    assert _prompt(lib, _shape(num_seqs=0), q=None) == OK
    for name in ("q", "k", "v", "start", "out"):
        assert _prompt(lib, s, **{name: None}) == INVALID
    for name in ("q", "k", "v", "out"):
        assert _prompt(lib, s, **{name: FAKE + 8}) == MISALIGNED
    assert _prompt(lib, s, start=FAKE + 2) == MISALIGNED
    for name, row in (("qs", 2048), ("ks", 1024), ("vs", 1024), ("os", 2048)):
        assert _prompt(lib, s, **{name: row - 8}) == INVALID
        assert _prompt(lib, s, **{name: row + 4}) == MISALIGNED
    assert _prompt(lib, s, vs=1 << 38) == UNSUPPORTED
    assert _prompt(lib, s, n=2 ** 31 - 1, longest=1) == UNSUPPORTED
    assert _prompt(lib, s, longest=2 ** 31 - 1) == UNSUPPORTED


@pytest.mark.parametrize("dtype", [W.DTYPE_F16, W.DTYPE_BF16])
@pytest.mark.parametrize("keys", [True, False])
def test_oracle_round_trip(dtype, keys):
    """store_row and load_rows agree on the layout, and a value is off by half a step at most."""
    rng = np.random.default_rng(3)
    d, hkv = 64, 2
    pool = np.full((3, hkv, I.record_bytes(d)), 0xFF, dtype=np.uint8)
    rows = I.narrow(rng.standard_normal((21, hkv, d)), dtype)
    codes, step, lo = I.quantise(rows, dtype)
    for j in range(21):
        for h in range(hkv):
            I.store_row(pool, keys, d, [2, 0][j // 16], h, j % 16, codes[j, h], step[j, h], lo[j, h])
    got = I.load_rows(pool, keys, d, [2, 0], 21, dtype)
    want = I.to_f64(rows, dtype).transpose(1, 0, 2)
    half = I.to_f64(step, dtype).T[..., None] / 2
    # the step's own rounding moves the top code by 15 x half a unit of it
    assert (np.abs(got - want) <= half * (1 + 30 * I.EPS[dtype])).all()
    built = I.build_pools(5, contexts=[21], hkv=hkv, d=d, dtype=dtype)
    back = I.load_rows(built[0 if keys else 1], keys, d, built[2][0], 21, dtype)
    assert np.isfinite(back).all() and np.abs(back).max() > 1


def test_calls_convert_their_arguments(lib):
    """The entry points of the compiled binding: what it takes for an address, a number and a
    structure, and what it refuses; num_tokens 0 launches nothing."""
    shape, axes = _shape(), P.RopeAxes.make([64])

    def call(q=FAKE, tokens=0, eps=1e-6, weight=None, sh=shape, ax=axes, stream=0):
        P.photon_qk_norm_rope(q, 0, FAKE, np.int64(0), weight, FAKE, eps, FAKE, FAKE, 16, ax,
                              tokens, FAKE2, 0, FAKE2, 0, sh, stream)

    class Held:
        def data_ptr(self):
            return FAKE

    for ok in (dict(), dict(q=Held()), dict(q=None), dict(q=2 ** 64 - 16), dict(tokens=np.int32(0)),
               dict(tokens=0.0), dict(eps=1), dict(eps=np.float32(0.5)), dict(weight=Held())):
        call(**ok)
    for error, bad in ((AttributeError, dict(q="address")), (OverflowError, dict(q=2 ** 64)),
                       (OverflowError, dict(tokens=2 ** 31)), (OverflowError, dict(tokens=-2 ** 31 - 1)),
                       (TypeError, dict(tokens=None)), (TypeError, dict(eps=None)),
                       (TypeError, dict(sh=None)), (TypeError, dict(sh=axes)),
                       (TypeError, dict(ax=bytes(3))), (AttributeError, dict(stream="s"))):
        with pytest.raises(error):
            call(**bad)
    with pytest.raises(P.PhotonError) as e:
        call(eps=float("inf"))
    assert e.value.status == INVALID
    with pytest.raises(OverflowError):     # a workspace's size has no sign
        P.photon_paged_decode_int4(FAKE, FAKE, FAKE, FAKE, FAKE, 0.1, FAKE2, FAKE, -1, shape, 0)
    native = P._native()
    with pytest.raises(TypeError):
        native.photon_qk_norm_rope(1, 2)
    with pytest.raises(ValueError):
        native.bind("photon_other", 1)

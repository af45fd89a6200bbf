"""8-bit caches without a GPU: what the calls refuse on the host, the rotary frequencies, and the references' own
consistency."""
import ctypes
import math

import pytest
import torch

from tests import _q8 as Q
from tests.test_abi_cpu import FAKE, good_dims, lib  # noqa: F401  (fixture)

ODD = ctypes.c_void_p(0x1008)
P = ctypes.c_void_p


class Cache(ctypes.Structure):
    _fields_ = [(n, P) for n in ("k", "k_scale", "v", "v_scale", "kidx", "kidx_scale")]


class Rows(ctypes.Structure):
    _fields_ = ([(n, P) for n in ("q", "k", "v", "q_idx", "k_idx")]
                + [(n + "_stride", ctypes.c_int64) for n in ("q", "k", "v", "q_idx", "k_idx")])


class Rope(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int32), ("rot_idx", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("gain", ctypes.c_float), ("inv_freq", P), ("inv_freq_idx", P)]


def cache(**kw):
    return Cache(**{**{n: 0x1000 for n, _ in Cache._fields_}, **kw})


def rows(**kw):
    d = {n: 0x1000 for n in ("q", "k", "v", "q_idx", "k_idx")}
    d.update(q_stride=8192, k_stride=1024, v_stride=1024, q_idx_stride=512, k_idx_stride=512)
    return Rows(**{**d, **kw})


def rope(**kw):
    return Rope(**{**dict(rot=64, rot_idx=64, interleaved=0, gain=1.0, inv_freq=0x1000, inv_freq_idx=0x1000), **kw})


def _append(lib, d, r=None, o=None, n_rows=8, n_req=2, n_pages=10, q_out=FAKE, kidx=FAKE):
    return lib.msa_rope_append(ctypes.byref(r or rows()), ctypes.byref(o or rope()), FAKE, FAKE, FAKE, n_rows, n_req,
                               n_pages, ctypes.byref(d), q_out, FAKE, FAKE, FAKE, kidx, FAKE, None)


def _append8(lib, d, r=None, o=None, n_rows=8, n_req=2, n_pages=10, q_out=FAKE, c=None):
    return lib.msa_rope_append_q8(ctypes.byref(r or rows()), ctypes.byref(o or rope()), FAKE, FAKE, FAKE, n_rows, n_req,
                                  n_pages, ctypes.byref(d), q_out, FAKE, ctypes.byref(c or cache()), FAKE, None)


def _read(lib, d, c=None, n_req=2, n_pages=10, n_out=10, k=FAKE, kidx=FAKE):
    return lib.msa_cache_read_q8(ctypes.byref(c or cache()), FAKE, FAKE, FAKE, n_req, n_pages, n_out, ctypes.byref(d), k,
                                 FAKE, kidx, FAKE, None)


def _score(lib, d, c=None, n_rows=8, n_req=2, n_pages=10, q=FAKE):
    return lib.msa_index_score_q8(q, ctypes.byref(c or cache()), FAKE, FAKE, FAKE, n_rows, n_req, n_pages,
                                  ctypes.byref(d), FAKE, FAKE, None)


def _attn(lib, d, c=None, B=8, n_pages=10, q=FAKE, out=FAKE):
    return lib.msa_sparse_attn_decode_q8(q, ctypes.byref(c or cache()), FAKE, FAKE, B, n_pages, ctypes.byref(d), out, FAKE,
                                         FAKE, None)


def _step(lib, d, c=None, B=8, n_pages=10, q=FAKE):
    return lib.msa_decode_step_q8(q, FAKE, ctypes.byref(c or cache()), FAKE, FAKE, B, n_pages, ctypes.byref(d),
                                  *([FAKE] * 7), None)


def _window(lib, d, c=None, n_rows=8, n_req=2, n_pages=10, window=128, n_sink=4, phase=0, q=FAKE, out=FAKE):
    return lib.msa_window_attn_q8(q, ctypes.byref(c or cache()), FAKE, FAKE, FAKE, n_rows, n_req, n_pages, window, n_sink,
                                  ctypes.byref(d), phase, out, FAKE, FAKE, None)


ALL = [_append, _append8, _read, _score, _attn, _step, _window]


@pytest.mark.parametrize("call", ALL)
@pytest.mark.parametrize("kw,status", [(dict(page_size=64), 2), (dict(topk=0), 1), (dict(max_blocks=0), 1),
                                       (dict(Hq=63), 1)])
def test_bad_dims(lib, call, kw, status):  # noqa: F811
    assert call(lib, good_dims(**kw)) == status


def test_unsupported_shapes(lib):  # noqa: F811
    for call in (_append, _append8, _read, _attn, _step, _window):
        assert call(lib, good_dims(D=96)) == 2 and call(lib, good_dims(Hq=16, G=8)) == 2
    for call in (_append, _append8, _read, _score, _step):
        assert call(lib, good_dims(Di=48)) == 2 and call(lib, good_dims(G=3, Hq=24)) == 2
    assert _step(lib, good_dims(max_blocks=16385)) == 2 and _step(lib, good_dims(), B=8192) == 2
    assert _window(lib, good_dims(max_blocks=(1 << 24) + 1)) == 2


def test_bad_sizes_and_pointers(lib):  # noqa: F811
    d = good_dims()
    for call in (_append, _append8, _score, _window):
        assert call(lib, d, n_rows=-1) == 1 and call(lib, d, n_req=0) == 1
    for call in ALL:
        assert call(lib, d, n_pages=0) == 1
    assert _read(lib, d, n_req=-1) == 1 and _read(lib, d, n_out=0) == 1 and _read(lib, d, k=None) == 1
    assert _read(lib, d, k=ctypes.c_void_p(0x1010)) == 1 and _read(lib, d, kidx=ctypes.c_void_p(0x1010)) == 1
    assert _attn(lib, d, B=-1) == 1 and _step(lib, d, B=-1) == 1
    for call in (_score, _attn, _step, _window):
        assert call(lib, d, q=None) == 1 and call(lib, d, q=ODD) == 1
    assert _attn(lib, d, out=ODD) == 1 and _window(lib, d, out=ODD) == 1
    for call in (_append, _append8):
        assert call(lib, d, q_out=None) == 1 and call(lib, d, q_out=ODD) == 1
    for name in ("k", "k_scale", "v", "v_scale"):
        for call in (_append8, _read, _attn, _step, _window):
            assert call(lib, d, c=cache(**{name: None})) == 1, name
            assert call(lib, d, c=cache(**{name: 0x1004})) == 1, name
    for name in ("kidx", "kidx_scale"):
        for call in (_append8, _read, _score, _step):
            assert call(lib, d, c=cache(**{name: None})) == 1, name
            assert call(lib, d, c=cache(**{name: 0x1004})) == 1, name
    assert _append(lib, d, kidx=None) == 1


def test_append_refuses_rows_and_rotations(lib):  # noqa: F811
    d = good_dims()
    for call in (_append, _append8):
        for name in ("q", "k", "v", "q_idx", "k_idx"):
            assert call(lib, d, r=rows(**{name: None})) == 1, name          # one of a pair missing too
            assert call(lib, d, r=rows(**{name: 0x1004})) == 1, name
            assert call(lib, d, r=rows(**{name + "_stride": 8196})) == 1, name
            assert call(lib, d, r=rows(**{name + "_stride": 256})) == 1, name   # rows would overlap
        assert call(lib, d, o=rope(rot=8)) == 2 and call(lib, d, o=rope(rot_idx=24)) == 2
        assert call(lib, d, o=rope(rot=144)) == 1 and call(lib, d, o=rope(rot=-16)) == 1
        assert call(lib, d, o=rope(rot_idx=80)) == 1 and call(lib, d, o=rope(interleaved=2)) == 1
        assert call(lib, d, o=rope(inv_freq=None)) == 1 and call(lib, d, o=rope(inv_freq_idx=None)) == 1


def test_window_refuses(lib):  # noqa: F811
    d = good_dims()
    assert _window(lib, d, window=0) == 1 and _window(lib, d, n_sink=-1) == 1 and _window(lib, d, phase=2) == 1
    assert _window(lib, d, n_rows=(1 << 23) + 1) == 2 and _attn(lib, d, B=(1 << 23) + 1) == 2
    assert _read(lib, good_dims(max_blocks=1 << 20), n_req=4096) == 2
    assert _score(lib, good_dims(max_blocks=1 << 20), n_rows=4096, n_req=4096) == 2


def test_nothing_to_do(lib):  # noqa: F811
    d = good_dims()
    assert _append(lib, d, n_rows=0) == 0 and _append8(lib, d, n_rows=0) == 0 and _read(lib, d, n_req=0) == 0
    assert _score(lib, d, n_rows=0) == 0 and _attn(lib, d, B=0) == 0 and _step(lib, d, B=0) == 0
    assert _window(lib, d, n_rows=0) == 0


def test_binding_refuses_before_the_call():
    import block_sparse_attention_06_gb300 as m
    dims = m.Dims(16, 2, 128, 64, 4, 3)
    c = m.CacheQ8.zeros(dims, 4, "cpu")
    assert c.k.dtype == torch.float8_e4m3fn and c.k_scale.dtype == torch.float8_e8m0fnu
    assert float(c.kidx_scale.float().min()) == 1.0
    q, i = torch.zeros(1, 16, 128, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    bt = torch.zeros(1, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        m.msa_window_attn_q8(q, c, bt, i, i, 4, 0, dims, m.MSA_PHASE_DECODE)
    with pytest.raises(ValueError, match="CUDA tensor"):
        m.msa_sparse_attn_decode_q8(q, c, i, i, dims)
    with pytest.raises(ValueError, match="CUDA tensor"):
        m.msa_cache_read_q8(c, bt, bt, i, dims, q, q)
    with pytest.raises(ValueError, match="multiples of 16"):
        m.Rope(24, torch.zeros(12, dtype=torch.float64))
    with pytest.raises(ValueError, match="CUDA"):
        m.Rope(16, torch.zeros(8, dtype=torch.float64))


def test_inv_freq():
    import block_sparse_attention_06_gb300 as m
    f, g = m.rope_inv_freq(64, 10000.0)
    assert g == 1.0 and f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([10000.0 ** (-2 * i / 64) for i in range(32)], dtype=torch.float64), rtol=1e-15)
    lin, _ = m.rope_inv_freq(64, scaling="linear", factor=8.0)
    assert torch.allclose(lin, f / 8, rtol=1e-15)
    ntk, _ = m.rope_inv_freq(64, scaling="ntk", factor=8.0)
    assert float(ntk[0]) == 1.0 and math.isclose(float(ntk[-1]), float(f[-1]) / 8, rel_tol=1e-12)
    yarn, gain = m.rope_inv_freq(64, scaling="yarn", factor=16.0, original_len=4096)
    assert math.isclose(gain, 0.1 * math.log(16.0) + 1)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(yarn[turns > 40], f[turns > 40])                      # fast pairs kept
    assert torch.allclose(yarn[turns < 0.8], f[turns < 0.8] / 16)            # slow pairs divided
    assert bool(((yarn <= f) & (yarn >= f / 16 * (1 - 1e-12))).all())
    assert m.rope_inv_freq(0)[0].numel() == 0
    for bad in (dict(rot=7), dict(rot=64, scaling="cubic"), dict(rot=64, factor=0.5), dict(rot=64, scaling="yarn")):
        with pytest.raises(ValueError):
            m.rope_inv_freq(**bad)


def test_reference_rounding_is_the_types():
    """The reference's own rounding against torch's e4m3 conversion, over all binades and ties."""
    x = torch.cat([torch.arange(-448, 449).double() / 512, torch.linspace(-448, 448, 20001).double(),
                   torch.tensor([1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0]).double()])
    step = Q.step_of(x)
    got = torch.round(x / step) * step
    assert torch.equal(got, x.float().to(torch.float8_e4m3fn).double())


def test_reference_scale_is_the_smallest_that_fits():
    amax = torch.tensor([0.0, 448.0, 448.0001, 449.0, 224.0, 224.1, 1.0, 0.875, 0.8751, 2.0 ** -130, 3.3e38]).double()
    assert Q.exponent(amax).tolist() == [0, 0, 1, 1, -1, 0, -8, -9, -8, -100, 120]
    code, e = Q.quantise(Q.f64(Q.normal((64, 32), 1)))
    top = code.abs().amax(-1)
    assert bool((top <= 448).all()) and bool((top >= 208).all())   # 224 rounded down by at most half a step


def test_stored_values_are_bf16_numbers():
    code, scale = Q.pages(2, 2, 32, 3)
    x = Q.stored(code, scale)
    assert torch.equal(x, Q.f64(x.to(torch.bfloat16)))


def test_reference_window_of_everything_is_dense_attention():
    bt, pool = Q.tables([200], 1)
    k, v = Q.stored(*Q.pages(pool, 2, 64, 2)), Q.stored(*Q.pages(pool, 2, 64, 3))
    q = Q.normal((3, 8, 64), 4)
    req, pos = torch.zeros(3).long(), torch.tensor([0, 57, 199])
    a = Q.ref_window(q, k, v, bt, req, pos, 1 << 30, 0, 0.125)
    b = Q.ref_window(q, k, v, bt, req, pos, 1, 200, 0.125)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    kk, vv = (x[bt[0].long()].transpose(0, 1).flatten(1, 2)[:, :200] for x in (k, v))
    for r in range(3):
        n = int(pos[r]) + 1
        o = torch.nn.functional.scaled_dot_product_attention(
            Q.f64(q[r]).reshape(2, 4, 64), kk[:, :n], vv[:, :n], scale=0.125).reshape(8, 64)
        assert torch.allclose(a[0][r], o, atol=1e-12)

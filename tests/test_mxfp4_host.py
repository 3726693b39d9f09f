"""The 4-bit (MXFP4) calls without a device: the reference of the GPU tests
against hand-worked values, and every refusal (nothing is launched: a call
that passes its checks would need pointers, which no test here gives)."""
import ctypes as C

import numpy as np
import pytest
import torch

import mxref
from compressed_sparse_kv_04_b200 import binding
from compressed_sparse_kv_04_b200 import build as csa_build


@pytest.fixture(scope="module")
def L():
    csa_build.build()
    return binding.lib()


def P(**kw):
    base = dict(B=2, d=512, H=128, H_I=64, D_I=128, k=1024, window=128, rope_dim=64, m=4)
    base.update(kw)
    return binding.make_params(**base)


def test_reference_rounds_ties_to_even_codes():
    x = np.zeros(32)
    x[:9] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -2.5]
    codes, s = mxref.quantise(x)
    assert s == [127]
    assert codes[:9].tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 12]
    assert mxref.values(codes, s)[:9].tolist() == [0, 1, 1, 2, 2, 4, 4, 6, -2]


def test_reference_scale_is_the_smallest_that_holds():
    for amax, e in ((6.0, 0), (6.03125, 1), (3.0, -1), (3.015625, 0), (448.0, 7), (2.0 ** -126, -127)):
        x = np.zeros(32)
        x[3] = -amax
        assert mxref.quantise(x)[1] == [e + 127], amax


def test_reference_values_are_exact_in_bf16():
    x = mxref.hard_rows(200, 128, 7)
    codes, s = mxref.quantise(mxref.bf16_values(x))
    v = mxref.values(codes, s)
    back = torch.from_numpy(v).bfloat16().double().numpy()
    assert np.array_equal(back[~np.isnan(v)], v[~np.isnan(v)])
    # no value saturates: half a step of the largest binade at most
    fin = np.isfinite(mxref.bf16_values(x)).reshape(200, -1, 32).all(-1)
    err = np.abs(v - mxref.bf16_values(x)).reshape(200, -1, 32).max(-1)
    assert (err[fin] <= np.exp2(s[fin].astype(float) - 127)).all()


def test_row_bytes(L):
    assert L.mxfp4_row_bytes(512) == 272 and L.mxfp4_row_bytes(128) == 80
    assert L.mxfp4_row_bytes(64) == 0 and L.mxfp4_row_bytes(-1) == 0
    with pytest.raises(binding.CsaError):
        binding.mxfp4_row_bytes(96)


def test_cache_write_refusals(L):
    def call(p, rows=None, stride=512, n=1, first=None, count=None, kv4=None, N=8):
        return L.mxfp4_cache_write(None if p is None else C.byref(p), rows, stride, n, first, count,
                                   kv4, N, None, None)
    assert call(None) == 1
    assert call(P(d=256)) == 2
    assert call(P(B=70000)) == 2
    assert call(P(), n=-1) == 1
    assert call(P(), N=0) == 1
    assert call(P(), N=1 << 31) == 1
    assert call(P(), n=0) == 0                      # nothing to do
    assert call(P()) == 1 and b"rows is null" in L.csa_last_error()
    assert call(P(), rows=8) == 1                   # alignment
    assert call(P(), rows=16, stride=520, n=2) == 1  # rows of two sequences overlap
    assert call(P(), rows=16, stride=516) == 1      # not a multiple of 8
    assert call(P(), rows=16, stride=-512) == 1
    assert call(P(), rows=16, first=4) == 1 and b"first_entry" in L.csa_last_error()
    assert call(P(), rows=16, count=12) == 1 and b"count" in L.csa_last_error()
    assert call(P(), rows=16) == 1 and b"kv4 is null" in L.csa_last_error()
    assert call(P(), rows=16, kv4=24) == 1


def test_cache_read_refusals(L):
    def call(p, kv4=None, N=8, idx=None, first=None, count=None, n=1, rows=None):
        return L.mxfp4_cache_read(None if p is None else C.byref(p), kv4, N, idx, first, count, n,
                                  rows, None, None)
    assert call(None) == 1
    assert call(P(d=64)) == 2
    assert call(P(), n=0) == 0
    assert call(P()) == 1 and b"kv4 is null" in L.csa_last_error()
    assert call(P(), kv4=16, idx=2) == 1
    assert call(P(), kv4=16, idx=16, first=16, rows=16) == 1
    assert b"exclude" in L.csa_last_error()
    assert call(P(), kv4=16) == 1 and b"rows is null" in L.csa_last_error()


def test_attention_refusals_name_the_4bit_cache(L):
    p = P()
    args = (16, 16, None, 8, 16, 16, 16, 8, 16, None, None, 16, None, None, 0, None, None)
    assert L.sparse_mqa_decode_mxfp4(C.byref(p), *args) == 1
    assert b"sparse_mqa_decode_mxfp4: kv4 is null" in L.csa_last_error()
    args = (16, 16, None, 8, 16, 8, 16, None, None, 16, None, None, 0, None, None)
    assert L.dense_mqa_decode_mxfp4(C.byref(p), *args) == 1
    assert b"dense_mqa_decode_mxfp4: kv4 is null" in L.csa_last_error()
    for kw in (dict(H=129), dict(rope_dim=63), dict(window=1025)):
        p = P(**kw)
        assert L.dense_mqa_decode_mxfp4(C.byref(p), *args) == 2, kw
    p = P()
    args = (16, 16, 16, 8, 16, 8, 16, None, None, 16, None, None, 0, None, None)
    assert L.dense_mqa_decode_mxfp4(C.byref(p), *args) == 4  # no workspace


def test_binding_checks_shapes_before_the_library():
    p = P(d=128, rope_dim=32)
    rows = torch.zeros(2, 3, 128, dtype=torch.bfloat16)
    kv4 = torch.zeros(2, 8, 80, dtype=torch.uint8)
    with pytest.raises(ValueError):
        binding.mxfp4_cache_write(p, rows, kv4)                    # host tensors
    with pytest.raises(ValueError):
        binding.mxfp4_cache_write(p, rows.float(), kv4)
    with pytest.raises(ValueError):
        binding.mxfp4_cache_write(p, rows[:, :, :64], kv4)
    with pytest.raises(ValueError):
        binding.mxfp4_cache_write(p, rows.transpose(0, 1), kv4)
    with pytest.raises(ValueError):
        binding.mxfp4_cache_read(p, kv4, rows.float())
    with pytest.raises(ValueError):
        binding.mxfp4_cache_read(p, kv4[:, :, :72], rows)
    with pytest.raises(TypeError):
        binding.mxfp4_cache_read(p, kv4, None)


def test_scale_bytes_and_quantize_refusals(L):
    assert L.mxfp4_scale_bytes(1, 128) == 512
    assert L.mxfp4_scale_bytes(129, 256) == 2 * 2 * 512
    for rows, cols in ((0, 128), (1, 96), (1, 0), (-1, 128), (65535 * 128 + 1, 128), (1, 1 << 25)):
        assert L.mxfp4_scale_bytes(rows, cols) == 0, (rows, cols)

    def call(rows=2, cols=256, x=None, ld=256, codes=None, scales=None):
        return L.mxfp4_quantize(rows, cols, x, ld, codes, scales, None)
    assert call(rows=0) == 0
    assert call(rows=-1) == 2
    assert call(cols=200) == 2
    assert call(ld=128) == 1
    assert call(ld=260) == 1
    assert call() == 1 and b"x is null" in L.csa_last_error()
    assert call(x=8) == 1
    assert call(x=16) == 1 and b"codes is null" in L.csa_last_error()
    assert call(x=16, codes=16) == 1 and b"scales is null" in L.csa_last_error()


def test_projection_refusals(L):
    ok = (8, 16, 128, 4, 128, 256)
    assert L.grouped_out_proj_mxfp4_workspace_bytes(*ok) > 0
    bad = [((0, 16, 128, 4, 128, 256), 1), ((8, 16, 128, 3, 128, 256), 2),
           ((8, 16, 128, 4, 64, 256), 2), ((8, 16, 128, 4, 128, 200), 2),
           ((8, 1, 128, 1, 256, 256), 2),         # (H/g)*D = 128
           ((8, 16, 128, 1, 128, 256), 2),        # g*d_g = 128
           ((65535 * 128 + 1, 16, 128, 4, 128, 256), 2)]
    null = (None,) * 8 + (0, None, None)
    for sizes, code in bad:
        assert L.grouped_out_proj_mxfp4_workspace_bytes(*sizes) == 0, sizes
        assert L.grouped_out_proj_mxfp4(*sizes, *null) == code, sizes
    assert L.grouped_out_proj_mxfp4(*ok, *null) == 1 and b"o is null" in L.csa_last_error()
    p = (16, 16, 16, 16, 16, None, 16)
    assert L.grouped_out_proj_mxfp4(*ok, *p, None, 0, None, None) == 4   # no workspace
    assert L.grouped_out_proj_mxfp4(*ok, *p, 16, 100, None, None) == 4   # too small
    assert L.grouped_out_proj_mxfp4(*ok, *p, 8, 1 << 40, None, None) == 1  # misaligned
    with pytest.raises(ValueError):
        binding.grouped_out_proj_mxfp4(torch.zeros(2, 3), None, None, None, None, None)


def test_workspace_is_checked_like_every_tensor():
    """On the host, and of another type: refused before the library sees it."""
    with pytest.raises(ValueError, match="ws is on cpu"):
        binding._ws(binding._device(), torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(TypeError, match="ws"):
        binding._ws(binding._device(), 16)
    assert binding._ws(binding._device(), None) == (None, 0)


def test_native_calls_check_every_argument():
    """Wrong types, shapes and places, each named; the library is not reached."""
    p = P(B=2, d=128, H=4, rope_dim=32, k=8)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    q, kv4, tok = bf(2, 4, 128), torch.zeros(2, 8, 80, dtype=torch.uint8), bf(2, 9, 128)
    pos, sink, out = torch.zeros(2, dtype=torch.int64), torch.zeros(4), bf(2, 4, 128)
    idx, cnt = torch.zeros(2, 8, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    dense = dict(p=p, q=q, pos_q=pos, kv4=kv4, kv_tok=tok, sink=sink, out=out)
    sparse = dict(dense, topk_idx=idx, topk_cnt=cnt)
    bad = [("q", bf(2, 4, 64), ValueError), ("q", 3, TypeError), ("kv4", None, TypeError),
           ("kv4", torch.zeros(2), ValueError), ("kv_tok", None, TypeError),
           ("q", torch.zeros(2, 4, 128), ValueError), ("p", kv4, TypeError)]
    for fn, args in ((binding.dense_mqa_decode_mxfp4, dense),
                     (binding.sparse_mqa_decode_mxfp4, sparse)):
        for name, value, error in bad:
            with pytest.raises(error, match=None if name == "p" else name):
                fn(**dict(args, **{name: value}))
        with pytest.raises(ValueError, match="q is on cpu"):
            fn(**args)
    with pytest.raises(binding.CsaError):
        binding.mxfp4_cache_read(P(d=256), kv4, bf(2, 3, 256))
    with pytest.raises(TypeError):
        binding._native().cache_write(p)


def test_native_projection_checks_every_argument():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    ok = dict(o=bf(2, 4, 128), w_g=u8(2, 128, 128), w_g_scale=u8(2 * 2 * 512), w_o=u8(256, 128),
              w_o_scale=u8(2 * 2 * 512), z=bf(2, 256), ws=u8(1 << 16))
    for name, value, error in (("o", bf(2, 4), ValueError), ("o", None, TypeError),
                               ("w_g", u8(2, 128), ValueError), ("w_o", None, TypeError),
                               ("z", bf(2, 255), ValueError)):
        with pytest.raises(error, match="o must be|is on cpu" if error is ValueError else name):
            binding.grouped_out_proj_mxfp4(**dict(ok, **{name: value}))
    with pytest.raises(ValueError, match="o is on cpu"):
        binding.grouped_out_proj_mxfp4(**ok)


class _FakeLib:
    """Every entry point returns success and is noted."""

    def __init__(self):
        self.reached = []

    def __getattr__(self, name):
        def call(*args):
            self.reached.append(name)
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    """The binding over a library that does nothing, tensors taken wherever they are."""
    lib = _FakeLib()
    monkeypatch.setattr(binding, "lib", lambda: lib)
    monkeypatch.setattr(binding, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(binding, "_stream", lambda stream=None: None)
    return lib


def _bf16_cache_calls(p, c):
    """Every call of the binding that takes a bf16 cache, on cache c."""
    x = torch.zeros(2, 9, 4)
    return {
        "hca_compress": lambda: binding.hca_compress(p, x, x, x, x, x, 0, 1, c),
        "csa_compress": lambda: binding.csa_compress(p, x, x, x, x, x, 0, 1, c),
        "sparse_mqa_decode": lambda: binding.sparse_mqa_decode(p, x, x, c, x, x, x, x, x),
        "dense_mqa_decode": lambda: binding.dense_mqa_decode(p, x, x, c, x, x, x),
        "csa_prefill_chunk": lambda: binding.csa_prefill_chunk(p, 0, 1, *[x] * 7, c, *[x] * 10),
        "hca_prefill_chunk": lambda: binding.hca_prefill_chunk(p, 0, 1, *[x] * 4, c, x, x, x),
        "csa_decode_step": lambda: binding.csa_decode_step(p, *[x] * 8, c, *[x] * 10),
        "hca_decode_step": lambda: binding.hca_decode_step(p, *[x] * 5, c, x, x, x),
        "sparse_mqa_partials": lambda: binding.sparse_mqa_partials(p, 1, x, x, c, *[x] * 5),
    }


def test_calls_on_bf16_caches_refuse_one_that_is_too_short(fake):
    """A 4-bit cache holds about a quarter of a bf16 cache's bytes: such a call
    would read and write past its end.  Refused before the library is reached."""
    p = P(B=2, k=8)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    for bad in (torch.zeros(2, 8, 272, dtype=torch.uint8), bf(2, 8, 511), bf(1, 8, 512)):
        for name, call in _bf16_cache_calls(p, bad).items():
            with pytest.raises(ValueError, match="kv_c holds"):
                call()
    assert fake.reached == []
    for name, call in _bf16_cache_calls(p, bf(2, 8, 512)).items():
        call()
    assert fake.reached == list(_bf16_cache_calls(p, None))


def test_prepared_steps_refuse_a_bf16_cache_that_is_too_short(fake):
    x, bad = torch.zeros(2, 9, 4), torch.zeros(1, 8, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="kv_c holds"):
        binding.CsaDecodeStep(P(B=2), *[x] * 7, bad, *[x] * 6)
    with pytest.raises(ValueError, match="kv_c holds"):
        binding.HcaDecodeStep(P(B=2), *[x] * 4, bad, x, x)


def test_bf16_projection_refuses_4bit_weights(fake):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    o, w_g, w_o, z, ws = bf(2, 4, 128), bf(2, 128, 256), bf(256, 256), bf(2, 256), u8(64)
    for bad in (dict(w_g=u8(2, 128, 128)), dict(w_o=u8(256, 128))):
        with pytest.raises(ValueError, match="mxfp4"):
            binding.grouped_out_proj(**dict(dict(o=o, w_g=w_g, w_o=w_o, z=z, ws=ws), **bad))
    assert fake.reached == []
    binding.grouped_out_proj(o, w_g, w_o, z, ws=ws)
    assert fake.reached == ["grouped_out_proj"]


def test_prepared_steps_take_a_bf16_cache_as_bytes(monkeypatch):
    """uint8 rows of d * 2 bytes are a bf16 cache, as before there were 4-bit
    ones; uint8 rows of the 4-bit width go to the 4-bit step."""
    monkeypatch.setattr(binding, "_ptr", lambda t: None if t is None else t.data_ptr())
    tok, x = torch.zeros(2, 9, 512, dtype=torch.bfloat16), torch.zeros(2, 9, 4)
    as_bytes = torch.zeros(2, 8, 512, dtype=torch.bfloat16).view(torch.uint8)
    csa = binding.CsaDecodeStep(P(B=2), tok, *[x] * 6, as_bytes, *[x] * 6)
    hca = binding.HcaDecodeStep(P(B=2), tok, *[x] * 3, as_bytes, x, x)
    assert csa._fn is binding.lib().csa_decode_step
    assert hca._fn is binding.lib().hca_decode_step
    with pytest.raises(ValueError, match="kv4 is on cpu"):
        binding.HcaDecodeStep(P(B=2), tok, *[x] * 3, torch.zeros(2, 8, 272, dtype=torch.uint8), x, x)
    with pytest.raises(ValueError, match="kv_c holds"):
        binding.HcaDecodeStep(P(B=2), tok, *[x] * 3, torch.zeros(2, 8, 80, dtype=torch.uint8), x, x)


def test_allocations_honour_device_zero(monkeypatch):
    """device=0 means device 0 where another device is current."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    placed = []
    monkeypatch.setattr(torch, "zeros", lambda *s, dtype=None, device=None: placed.append(device))
    for device in (0, "cuda:2", None):
        binding.mxfp4_cache(P(), 8, device=device)
        binding.workspace(P(), binding.OP_DENSE_MQA, 1, 8, device=device)
    assert placed == [0, 0, "cuda:2", "cuda:2", 1, 1]

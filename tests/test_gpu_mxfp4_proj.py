"""GPU tests of the grouped output projection in 4 bits (MXFP4) and of its
operands.

Operands are compared bit for bit with the 64-bit reference.  Products: the
E2M1 values and their power-of-two scales multiply exactly, so y differs from
the 64-bit sum by fp32 accumulation and one bf16 rounding (half a step,
2^-8 relative): |d| <= 2^-8 |y| + A.  A bounds the accumulation: each of K
additions errs by at most 2^-24 of a partial sum, itself at most
S = sum |w| |x|, and the tensor cores may truncate where fp32 rounds (one more
bit): A = K * 2^-23 * S, far above what is seen and far below a lost term.
z is checked against the products of the library's own y, quantised by the
reference (so that no bf16 rounding of y stands between the two)."""
import numpy as np
import pytest
import torch

import mxref
from compressed_sparse_kv_04_b200 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    binding.lib()


def operand(w):
    """(codes, scale tiles, fp64 values) of a bf16 matrix, by the library."""
    codes, scales = binding.mxfp4_quantize(w)
    return codes, scales, values(codes, scales)


def values(codes, scales):
    """fp64 values of an operand, decoded on the device (large weights)."""
    rows, half = codes.shape
    nb = half * 2 // 32
    r = torch.arange(rows, device=DEV)[:, None]
    k = torch.arange(nb, device=DEV)[None]
    at = ((r // 128) * (nb // 4) + k // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + k % 4
    s = torch.exp2(scales.flatten()[at].double() - 127)
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(rows, -1).long()
    grid = torch.tensor(list(mxref.GRID) + list(-mxref.GRID), dtype=torch.float64, device=DEV)
    return grid[c] * s.repeat_interleave(32, 1)


@pytest.mark.parametrize("rows,cols", [(1, 128), (7, 256), (128, 384), (130, 128), (300, 1024)])
def test_operand_bytes(rows, cols):
    x = mxref.hard_rows(rows, cols, rows + cols)
    codes, scales = binding.mxfp4_quantize(x.to(DEV))
    torch.cuda.synchronize()
    rc, rs = mxref.quantise(mxref.bf16_values(x))
    assert np.array_equal(codes.cpu().numpy(), mxref.pack(rc))
    assert np.array_equal(scales.cpu().numpy(), mxref.scale_tiles(rs).reshape(-1))


def test_operand_of_a_slice():
    x = mxref.hard_rows(20, 512, 3).to(DEV)
    a = binding.mxfp4_quantize(x[3:14, 128:384])
    b = binding.mxfp4_quantize(x[3:14, 128:384].contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


class Layer:
    def __init__(self, H, D, g, d_g, d_model, seed):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.H, self.D, self.g, self.d_g, self.d_model = H, D, g, d_g, d_model
        k1 = H // g * D
        wg = (torch.randn(g * d_g, k1, generator=gen, device=DEV) / k1 ** 0.5).bfloat16()
        wo = (torch.randn(d_model, g * d_g, generator=gen, device=DEV) / (g * d_g) ** 0.5).bfloat16()
        self.w_g, self.w_gs, self.vg = operand(wg)
        self.w_o, self.w_os, self.vo = operand(wo)
        self.w_g = self.w_g.view(g, d_g, k1 // 2)
        self.gen = gen

    def tokens(self, T):
        return (torch.randn(T, self.H, self.D, generator=self.gen, device=DEV) *
                torch.rand(T, 1, 1, generator=self.gen, device=DEV) * 3).bfloat16()

    def run(self, o, with_y=True, ws=None):
        T = o.shape[0]
        y = torch.full((T, self.g * self.d_g), float("nan"), dtype=torch.bfloat16, device=DEV)
        z = torch.full((T, self.d_model), float("nan"), dtype=torch.bfloat16, device=DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        binding.grouped_out_proj_mxfp4(o, self.w_g, self.w_gs, self.w_o, self.w_os, z,
                                       y=y if with_y else None, ws=ws, dev_status=st)
        torch.cuda.synchronize()
        assert st.item() == 0, st.item()
        return y, z

    def check(self, o, y, z, rows=None):
        T = o.shape[0]
        rows = torch.arange(T, device=DEV) if rows is None else torch.tensor(rows, device=DEV)
        k1, d_g = self.H // self.g * self.D, self.d_g
        x = o[rows].reshape(len(rows), -1)
        xq = values(*binding.mxfp4_quantize(x))
        for j in range(self.g):
            a, w = xq[:, j * k1: (j + 1) * k1], self.vg[j * d_g: (j + 1) * d_g]
            self.close(y[rows, j * d_g: (j + 1) * d_g], a, w)
        yq = values(*binding.mxfp4_quantize(y[rows].contiguous()))
        self.close(z[rows], yq, self.vo)

    @staticmethod
    def close(got, a, w):
        ref, mag = a @ w.T, a.abs() @ w.abs().T
        err = (got.double() - ref).abs()
        bound = ref.abs() * 2.0 ** -8 + mag * (a.shape[1] * 2.0 ** -23)
        assert torch.isfinite(got).all()
        assert (err <= bound).all(), (err - bound).max().item()


@pytest.mark.parametrize("T", [1, 3, 16, 17, 33, 64, 65, 128, 129, 200, 300])
def test_small(T):
    """Every tile form: one token to several token tiles."""
    m = Layer(16, 128, 4, 128, 256, T)
    o = m.tokens(T)
    y, z = m.run(o)
    m.check(o, y, z)


@pytest.mark.parametrize("H,D,g,d_g,d_model", [
    (2, 128, 1, 256, 128),     # one group, the smallest inner dimension
    (16, 512, 2, 128, 128),    # long inner dimension, few tiles: K splits
    (12, 512, 3, 512, 640),    # odd tile counts; 640 = 2.5 tiles of 256
    (8, 512, 2, 384, 384),     # neither product has whole tiles of 256
    (64, 512, 16, 512, 5120),
])
@pytest.mark.parametrize("T", [5, 130, 520])
def test_shapes(H, D, g, d_g, d_model, T):
    m = Layer(H, D, g, d_g, d_model, 7)
    o = m.tokens(T)
    y, z = m.run(o)
    m.check(o, y, z)


@pytest.mark.parametrize("T", [8, 100, 1000, 4096])
def test_large_layer(T):
    """The V4-Pro projection (16 groups of 8 heads of 512)."""
    m = Layer(128, 512, 16, 1024, 7168, 1)
    o = m.tokens(T)
    y, z = m.run(o)
    rng = np.random.default_rng(T)
    rows = sorted({0, T - 1, T // 2, *rng.choice(T, min(T, 40), replace=False).tolist()})
    m.check(o, y, z, rows)


def test_wide_range_of_scales():
    """Tokens from 2^-100 to 2^100: the block scales carry the range."""
    m = Layer(16, 128, 4, 128, 256, 2)
    for T in (9, 260):
        o = m.tokens(T)
        o = (o.float() * torch.exp2(torch.linspace(-100, 100, T, device=DEV).round())[:, None, None])
        o = o.bfloat16()
        y, z = m.run(o)
        m.check(o, y, z)


def test_zero_and_nan_tokens():
    """A zero token gives zeros; NaN or infinity in a token stays in it."""
    m = Layer(16, 128, 4, 128, 256, 3)
    for T in (9, 260):
        o = m.tokens(T)
        o[2] = 0
        ref_y, ref_z = m.run(o)
        assert (ref_y[2] == 0).all() and (ref_z[2] == 0).all()
        bad = o.clone()
        bad[5, 0, 3] = float("nan")
        bad[7, 15, 127] = float("inf")
        y, z = m.run(bad)
        keep = torch.ones(T, dtype=torch.bool, device=DEV)
        keep[5] = keep[7] = False
        assert torch.equal(y[keep], ref_y[keep]) and torch.equal(z[keep], ref_z[keep])
        assert torch.isnan(y[5, :128]).all() and torch.equal(y[5, 128:], ref_y[5, 128:])
        assert torch.isnan(y[7, 384:]).all() and torch.equal(y[7, :384], ref_y[7, :384])
        assert torch.isnan(z[5]).all() and torch.isnan(z[7]).all()


@pytest.mark.parametrize("T", [6, 150])
def test_without_y_dirty_workspace_and_repeats(T):
    """y kept inside gives the same z; workspace contents do not matter; the
    call repeats bit for bit, also captured, on another stream."""
    m = Layer(16, 128, 4, 128, 256, 4)
    o = m.tokens(T)
    n = binding.grouped_out_proj_mxfp4_workspace_bytes(T, 16, 128, 4, 128, 256)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    y, z = m.run(o, ws=ws)
    m.check(o, y, z)
    _, z2 = m.run(o, with_y=False, ws=ws.fill_(0x7F))
    assert torch.equal(z, z2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    z3 = torch.empty_like(z)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        binding.grouped_out_proj_mxfp4(o, m.w_g, m.w_gs, m.w_o, m.w_os, z3, ws=ws)
    for _ in range(3):
        z3.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, z3)


def test_rows_behind_the_last_token_are_left():
    m = Layer(16, 128, 4, 128, 256, 5)
    for T in (3, 131):
        o = m.tokens(T)
        y = torch.full((T + 5, 512), 7.0, dtype=torch.bfloat16, device=DEV)
        z = torch.full((T + 5, 256), 7.0, dtype=torch.bfloat16, device=DEV)
        binding.grouped_out_proj_mxfp4(o, m.w_g, m.w_gs, m.w_o, m.w_os, z[:T], y=y[:T])
        torch.cuda.synchronize()
        assert (y[T:] == 7).all() and (z[T:] == 7).all()
        m.check(o, y[:T], z[:T])


def test_two_streams_two_workspaces():
    """Calls of every form at once, each with its own workspace, repeat what
    they give alone."""
    m = Layer(64, 512, 8, 1024, 4096, 6)
    tokens = [m.tokens(T) for T in (8, 200, 700)]
    alone = [m.run(o, with_y=False)[1] for o in tokens]
    ws = [torch.empty(binding.grouped_out_proj_mxfp4_workspace_bytes(o.shape[0], 64, 512, 8, 1024,
                                                                     4096),
                      dtype=torch.uint8, device=DEV) for o in tokens]
    z = [torch.empty_like(a) for a in alone]
    streams = [torch.cuda.Stream() for _ in tokens]
    torch.cuda.synchronize()
    for _ in range(4):
        for o, w, out, s in zip(tokens, ws, z, streams):
            binding.grouped_out_proj_mxfp4(o, m.w_g, m.w_gs, m.w_o, m.w_os, out, ws=w, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(alone, z):
        assert torch.equal(a, b)


def test_memory_of_a_call_belongs_to_its_stream():
    """Operands and workspace that a call on another stream allocates itself:
    freed and allocated again at once on the current stream, they are not
    written to before the call has read them."""
    T, H, D, g, d_g, d_model = 200, 32, 512, 4, 512, 1024
    gen = torch.Generator(device=DEV).manual_seed(5)
    o = torch.randn(T, H, D, generator=gen, device=DEV).bfloat16()
    wg = torch.randn(g * d_g, H // g * D, generator=gen, device=DEV).bfloat16()
    wo = torch.randn(d_model, g * d_g, generator=gen, device=DEV).bfloat16()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    wgc, wgs = binding.mxfp4_quantize(wg, stream=s)
    woc, wos = binding.mxfp4_quantize(wo, stream=s)
    wgc = wgc.view(g, d_g, -1)
    z = torch.empty(T, d_model, dtype=torch.bfloat16, device=DEV)
    want = torch.empty_like(z)
    s.synchronize()
    binding.grouped_out_proj_mxfp4(o, wgc, wgs, woc, wos, want)
    torch.cuda.synchronize()
    n = binding.grouped_out_proj_mxfp4_workspace_bytes(T, H, D, g, d_g, d_model)
    for _ in range(20):
        z.zero_()
        s.wait_stream(torch.cuda.current_stream())
        binding.grouped_out_proj_mxfp4(o, wgc, wgs, woc, wos, z, stream=s)
        torch.empty(n, dtype=torch.uint8, device=DEV).fill_(255)
        torch.cuda.synchronize()
        assert torch.equal(z, want)


def test_no_rows():
    codes, scales = binding.mxfp4_quantize(torch.zeros(0, 256, dtype=torch.bfloat16, device=DEV))
    assert codes.shape == (0, 128) and scales.numel() == 0

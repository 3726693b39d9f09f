"""GPU tests of the 4-bit (MXFP4) compressed cache: writing and reading rows
(bit for bit against the 64-bit reference), and compression into it (the bytes
of the bf16 entries, quantised)."""
import numpy as np
import pytest
import torch

import mxref
from compressed_sparse_kv_04_b200 import binding, configs, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    binding.lib()


def i64(*v):
    return torch.tensor(v, dtype=torch.int64, device=DEV)


def written(rows, n_cap, first, count, fill=0xAB):
    """The cache after the write, by the reference: untouched bytes keep `fill`."""
    B, n, d = rows.shape
    out = np.full((B, n_cap, mxref.row_bytes(d)), fill, np.uint8)
    for b in range(B):
        for i in range(max(0, min(count[b], n))):
            if 0 <= first[b] + i < n_cap:
                out[b, first[b] + i] = mxref.cache_rows(mxref.bf16_values(rows[b, i]), fill)
    return out


@pytest.mark.parametrize("d", [128, 512])
@pytest.mark.parametrize("B,n,n_cap,first,count", [
    (1, 1, 1, [0], [1]),
    (1, 700, 700, [0], [700]),
    (3, 37, 64, [0, 27, 13], [37, 37, 5]),
    (4, 17, 40, [3, 0, 23, 9], [0, -4, 17, 99]),   # nothing, nothing, all, clamped to n
])
def test_write_bytes(d, B, n, n_cap, first, count):
    rows = mxref.hard_rows(B * n, d, 11 + d + n).view(B, n, d)
    kv4 = torch.full((B, n_cap, binding.mxfp4_row_bytes(d)), 0xAB, dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    p = binding.make_params(B, d)
    binding.mxfp4_cache_write(p, rows.to(DEV), kv4, first_entry=i64(*first), count=i64(*count),
                              dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    assert np.array_equal(kv4.cpu().numpy(), written(rows, n_cap, first, count))


@pytest.mark.parametrize("d", [128, 512])
def test_write_defaults_and_strided_rows(d):
    """No first entries and no counts; rows that are a slice of a longer buffer."""
    B, n, n_cap = 3, 21, 30
    big = mxref.hard_rows(B * 40, d, 5).view(B, 40, d).to(DEV)
    kv4 = binding.mxfp4_cache(binding.make_params(B, d), n_cap)
    binding.mxfp4_cache_write(binding.make_params(B, d), big[:, 7: 7 + n], kv4)
    torch.cuda.synchronize()
    ref = written(big[:, 7: 7 + n].cpu(), n_cap, [0] * B, [n] * B, fill=0)
    assert np.array_equal(kv4.cpu().numpy(), ref)


def test_write_outside_the_cache_is_skipped_and_reported():
    d, B, n, n_cap = 128, 4, 9, 12
    first = [-3, 8, 1 << 62, -(1 << 62)]
    rows = mxref.hard_rows(B * n, d, 3).view(B, n, d)
    kv4 = torch.full((B, n_cap, 80), 0xAB, dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    binding.mxfp4_cache_write(binding.make_params(B, d), rows.to(DEV), kv4,
                              first_entry=i64(*first), dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 7
    assert np.array_equal(kv4.cpu().numpy(), written(rows, n_cap, first, [n] * B))


@pytest.mark.parametrize("d", [128, 512])
def test_read_range_and_count(d):
    B, n, n_cap = 3, 33, 50
    p = binding.make_params(B, d)
    host = mxref.cache_rows(mxref.bf16_values(mxref.hard_rows(B * n_cap, d, 9))).reshape(B, n_cap, -1)
    first, count = [0, 17, 4], [33, 33, 11]
    out = torch.full((B, n, d), 7.0, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    binding.mxfp4_cache_read(p, torch.from_numpy(host).to(DEV), out, first_entry=i64(*first),
                             count=i64(*count), dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    got = mxref.bf16_values(out)
    for b in range(B):
        ref = mxref.cache_values(host[b, first[b]: first[b] + count[b]], d)
        assert np.array_equal(got[b, : count[b]], ref, equal_nan=True)
        assert (got[b, count[b]:] == 7.0).all()


@pytest.mark.parametrize("d", [128, 512])
def test_read_every_code_and_scale(d):
    """All 16 codes under all 256 scale bytes (255: NaN)."""
    n_cap = 256 * 32 // d * 4
    rb = binding.mxfp4_row_bytes(d)
    host = np.zeros((1, n_cap, rb), np.uint8)
    nb = n_cap * d // 32
    codes = (np.arange(nb * 32) % 16).astype(np.uint8).reshape(1, n_cap, d)
    host[..., : d // 2] = mxref.pack(codes)
    host[..., d // 2: d // 2 + d // 32] = (np.arange(nb) % 256).astype(np.uint8).reshape(1, n_cap, -1)
    out = torch.empty(1, n_cap, d, dtype=torch.bfloat16, device=DEV)
    binding.mxfp4_cache_read(binding.make_params(1, d), torch.from_numpy(host).to(DEV), out)
    torch.cuda.synchronize()
    ref = mxref.cache_values(host, d)
    # 2^127 and 2^126 times 4 and 6 leave the range of bf16.
    ref = torch.from_numpy(ref).bfloat16().double().numpy()
    assert np.array_equal(mxref.bf16_values(out), ref, equal_nan=True)


def test_read_indices():
    d, B, n, n_cap = 512, 2, 6, 20
    host = mxref.cache_rows(np.random.default_rng(1).standard_normal((B, n_cap, d)).astype(np.float16)
                            .astype(np.float64))
    idx = torch.tensor([[3, 3, -1, 19, 20, 0], [5, -2, 7, 7, 7, 11]], dtype=torch.int32, device=DEV)
    out = torch.full((B, n, d), 7.0, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    p = binding.make_params(B, d)
    binding.mxfp4_cache_read(p, torch.from_numpy(host).to(DEV), out, idx=idx, count=i64(6, 5),
                             dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 7  # entries 20 and -2 lie outside
    got, vals = mxref.bf16_values(out), mxref.cache_values(host, d)
    for b, row in enumerate([[3, 3, None, 19, None, 0], [5, None, 7, 7, 7, None]]):
        for i, e in enumerate(row):
            assert np.array_equal(got[b, i], np.full(d, 7.0) if e is None else vals[b, e]), (b, i)


def test_write_then_read_in_a_graph_on_another_stream():
    """The pair captured once and replayed on new rows, beside work on the
    default stream."""
    d, B, n = 512, 2, 5
    p = binding.make_params(B, d)
    rows = torch.zeros(B, n, d, dtype=torch.bfloat16, device=DEV)
    kv4 = binding.mxfp4_cache(p, 16)
    out = torch.zeros(B, n, d, dtype=torch.bfloat16, device=DEV)
    first = i64(2, 9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            binding.mxfp4_cache_write(p, rows, kv4, first_entry=first)
            binding.mxfp4_cache_read(p, kv4, out, first_entry=first)
    for seed in (1, 2):
        new = torch.randn(B, n, d, generator=torch.Generator().manual_seed(seed)).bfloat16()
        rows.copy_(new)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g.replay()
        s.synchronize()
        assert np.array_equal(mxref.bf16_values(out),
                              mxref.values(*mxref.quantise(mxref.bf16_values(new))))


@pytest.mark.parametrize("name,kw", [
    ("csa_decode_128k_b8", dict(B=3, L=301)),
    ("csa_decode_128k_b8", dict(B=2, L=130, overlap=4)),
    ("csa_decode_tiny_4k", dict(B=2, L=130)),
    ("hca_decode_1m_b8", dict(B=2, L=700)),
])
def test_compression_into_the_cache(name, kw):
    """The entries' bytes are those of the bf16 entries, quantised; indexer keys
    and scales are those of the bf16 call."""
    w = configs.scaled(configs.BY_NAME[name], **kw)
    B, N, m = w.B, w.N_c + 2, w.m
    kv_tok, idx_tok = synth.token_streams(w, device=DEV)
    w_s, b_pos = synth.pool_params(w, DEV)
    ctx = i64(*[w.L - 3 * b for b in range(B)])
    gamma = synth.gains(w.d, 4, DEV)
    p = binding.params_for(w)
    first, nb = 1, w.N_c - 1
    kv_c = torch.zeros(B, N, w.d, dtype=torch.bfloat16, device=DEV)
    kv4 = torch.full((B, N, binding.mxfp4_row_bytes(w.d)), 0xAB, dtype=torch.uint8, device=DEV)
    if w.csa:
        w_si, b_pi = synth.pool_params(w, DEV, indexer=True)
        keys = [(torch.zeros(B, N, w.D_I, dtype=torch.uint8, device=DEV),
                 torch.zeros(B, N, device=DEV)) for _ in range(2)]
        binding.csa_compress(p, kv_tok, ctx, w_s, b_pos, gamma, first, nb, kv_c, idx_tok, w_si, b_pi,
                             *keys[0])
        binding.csa_compress_mxfp4(p, kv_tok, ctx, w_s, b_pos, gamma, first, nb, kv4, idx_tok, w_si,
                                   b_pi, *keys[1])
        torch.cuda.synchronize()
        assert torch.equal(keys[0][0], keys[1][0]) and torch.equal(keys[0][1], keys[1][1])
    else:
        binding.hca_compress(p, kv_tok, ctx, w_s, b_pos, gamma, first, nb, kv_c)
        binding.hca_compress_mxfp4(p, kv_tok, ctx, w_s, b_pos, gamma, first, nb, kv4)
        torch.cuda.synchronize()
    got, bits = kv4.cpu().numpy(), mxref.bf16_values(kv_c)
    for b in range(B):
        n = min(first + nb, -(-int(ctx[b]) // m))  # blocks with a token
        assert np.array_equal(got[b, first:n], mxref.cache_rows(bits[b, first:n], 0xAB)), b
        assert (got[b, :first] == 0xAB).all() and (got[b, n:] == 0xAB).all()


def _captured(fn):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        fn(s)
    return g


def test_calls_behind_copies_memsets_and_joined_streams():
    """The calls' first kernels may be scheduled early: behind a memset, a copy, a
    kernel and a joined stream, eager and captured, they see what came before."""
    d, B, n, N = 512, 4, 300, 400
    gen = torch.Generator(device=DEV).manual_seed(11)
    p = binding.make_params(B, d)
    src = torch.randn(B, n, d, generator=gen, device=DEV).bfloat16()
    rows, back = torch.zeros_like(src), torch.zeros_like(src)
    kv4, copy = binding.mxfp4_cache(p, N), binding.mxfp4_cache(p, N)
    binding.mxfp4_cache_write(p, src, kv4)
    want = torch.empty_like(src)
    binding.mxfp4_cache_read(p, kv4, want)
    want4 = kv4.clone()
    side = torch.cuda.Stream()

    def chain(s):
        kv4.zero_()
        rows.copy_(src)
        binding.mxfp4_cache_write(p, rows, kv4)   # behind a copy
        copy.copy_(kv4)
        back.zero_()
        binding.mxfp4_cache_read(p, copy, back)   # behind a memset
        side.wait_stream(s)
        with torch.cuda.stream(side):
            rows.neg_()
            kv4.zero_()
        s.wait_stream(side)
        binding.mxfp4_cache_write(p, rows, kv4)   # behind a joined stream
        binding.mxfp4_cache_read(p, kv4, rows)    # behind a call

    def check():
        torch.cuda.synchronize()
        assert torch.equal(back, want)
        assert torch.equal(rows, -want)
        assert torch.equal(copy, want4)
        for t in (kv4, copy, back, rows):
            t.fill_(1)

    for _ in range(20):
        chain(torch.cuda.current_stream())
        check()
    g = _captured(chain)
    for _ in range(20):
        g.replay()
        check()


def test_values_next_to_the_largest_stay_finite():
    """Above 6 * 2^125 = 1.5 * 2^127 values are stored as that, not as infinity;
    the scale byte stays at 252, the largest whose every code is finite in bf16."""
    top = 1.5 * 2.0 ** 127
    mags = torch.tensor([1.5, 1.5078125, 1.625, 1.75, 1.875, 1.9921875]).double() * 2.0 ** 127
    rows = torch.zeros(1, len(mags), 128, dtype=torch.double)
    rows[0, :, 3] = mags
    rows[0, :, 40] = -mags
    rows[0, :, 41] = 2.0 ** 125  # code 2: the block's other values keep their step
    rows = rows.bfloat16().to(DEV)
    assert torch.equal(rows[0, :, 3].double().cpu(), mags)
    p = binding.make_params(1, 128)
    kv4 = binding.mxfp4_cache(p, len(mags))
    binding.mxfp4_cache_write(p, rows, kv4)
    back = torch.empty_like(rows)
    binding.mxfp4_cache_read(p, kv4, back)
    codes, scales = binding.mxfp4_quantize(rows[0])
    torch.cuda.synchronize()
    want = torch.zeros(1, len(mags), 128, dtype=torch.double)
    want[0, :, 3], want[0, :, 40], want[0, :, 41] = top, -top, 2.0 ** 125
    assert torch.equal(back.double().cpu(), want)
    assert kv4[0, :, 64].eq(252).all() and kv4[0, :, 65].eq(252).all()
    assert torch.equal(codes, kv4[0, :, :64])
    assert scales.view(32, 16)[: len(mags), :2].eq(252).all()

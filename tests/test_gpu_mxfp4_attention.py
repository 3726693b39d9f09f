"""GPU tests of the attention over a 4-bit (MXFP4) cache, against the fp64
oracle on the cache's stored values (exact in bf16, so the oracle takes them
as a bf16 cache).

Tolerance.  A rounding to bf16 is off by at most 2^-8 of the power of two below
the value, uniformly: 2^-8 / sqrt(3) of it in the mean square, and values
spread over a binade are 1.44 times it or more in the mean, so the output's
rounding alone stays below 2^-9 (relative, L2).  Four factors of every term
carry one fp16 rounding each, 2^-12 by the same count (query, window key and
value, weight, split partial).  Together: 2^-9 + 4 * 2^-12, about half of what
bf16 operands would need.  The log-sum-exp moves by the query's and the window
keys' fp16 rounding, at most 2 * 2^-11 scale |qhat| |o| + 1e-4 (the derivation
of gpuhelp.lse_tolerance with 2^-11 in place of 2^-8).
"""
import numpy as np
import pytest
import torch

import mxref
from compressed_sparse_kv_04_b200 import binding, configs, synth
from gpuhelp import attention_errors, bits16, f32, lse_tolerance

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    binding.lib()


def assert_close(out, lse, ref_out, ref_lse, gain=1.0, scale=None):
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert attention_errors(got, ref_out)[1] <= 2.0 ** -9 + 4 * 2.0 ** -12
    if lse is not None:
        scale = 1.0 / got.shape[-1] ** 0.5 if scale is None else scale
        tol = (lse_tolerance(ref_out, scale, gain) - 1e-4) / 8 + 1e-4
        fin = np.isfinite(ref_lse)
        l = f32(lse).astype(np.float64)
        assert np.array_equal(l[~fin], ref_lse[~fin])
        assert (np.abs(l - ref_lse)[fin] <= tol[fin]).all(), np.abs(l - ref_lse)[fin].max()


class Case:
    def __init__(self, B, d, H, R, W, m, pos, N_cap, k=0, seed=1, gains=False, scale=1.0,
                 offset=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.p = binding.make_params(B, d, H=H, k=k, window=W, rope_dim=R, m=m, entry_offset=offset)
        self.m, self.W, self.R, self.k = m, W, R, k
        rows = torch.randn(B, N_cap, d, generator=g, device=DEV)
        rows = (rows * rows.square().mean(-1, keepdim=True).rsqrt() * scale).bfloat16()
        self.kv4 = binding.mxfp4_cache(self.p, N_cap)
        binding.mxfp4_cache_write(self.p, rows, self.kv4)
        self.pos = torch.tensor(pos, dtype=torch.int64, device=DEV)
        L = max(pos) + 1
        self.kv_tok = torch.randn(B, L, d, generator=g, device=DEV).bfloat16()
        self.q = torch.randn(B, H, d, generator=g, device=DEV).bfloat16()
        self.sink = torch.randn(H, generator=g, device=DEV)
        self.gq = synth.gains(d, seed, DEV) if gains else None
        self.gkv = synth.gains(d, seed + 1, DEV) if gains else None
        self.sel = self.cnt = None
        if k:
            n_vis = [min(max((x + 1) // m - offset, 0), N_cap) for x in pos]
            rng = np.random.default_rng(seed)
            sel = np.full((B, k), -1, np.int32)
            for b, v in enumerate(n_vis):
                c = min(k, v)
                sel[b, :c] = np.sort(rng.choice(v, c, replace=False)) if c else []
            self.sel = torch.from_numpy(sel).to(DEV)
            self.cnt = torch.tensor([min(k, v) for v in n_vis], dtype=torch.int32, device=DEV)

    def values(self):
        """The cache's stored values as a bf16 cache."""
        out = torch.empty(*self.kv4.shape[:2], self.p.d, dtype=torch.bfloat16, device=DEV)
        binding.mxfp4_cache_read(self.p, self.kv4, out)
        return out

    def run(self, cache, status=0, ws=None):
        p, B = self.p, self.p.B
        out = torch.full((B, p.H, p.d), float("nan"), dtype=torch.bfloat16, device=DEV)
        lse = torch.full((B, p.H), float("nan"), device=DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        op = binding.OP_SPARSE_MQA if self.k else binding.OP_DENSE_MQA
        ws = binding.workspace(p, op, 1, cache.shape[1]) if ws is None else ws
        kw = dict(gamma_q=self.gq, gamma_kv=self.gkv, lse=lse, ws=ws, dev_status=st)
        if self.k:
            binding.sparse_mqa_decode_mxfp4(p, self.q, self.pos, cache, self.sel, self.cnt,
                                            self.kv_tok, self.sink, out, **kw)
        else:
            binding.dense_mqa_decode_mxfp4(p, self.q, self.pos, cache, self.kv_tok, self.sink, out,
                                           **kw)
        torch.cuda.synchronize()
        assert st.item() == status, st.item()
        return out, lse

    def oracle(self, orc):
        B, p = self.p.B, self.p
        ro, rl = orc.mqa(bits16(self.q).reshape(B, 1, p.H, p.d),
                         self.pos.cpu().numpy().reshape(B, 1), bits16(self.values()),
                         bits16(self.kv_tok), f32(self.sink), self.m, self.W, self.R,
                         None if self.sel is None else self.sel.cpu().numpy().reshape(B, 1, -1),
                         None if self.cnt is None else self.cnt.cpu().numpy().reshape(B, 1),
                         None if self.gq is None else f32(self.gq),
                         None if self.gkv is None else f32(self.gkv))
        return ro[:, 0], rl[:, 0]

    def check(self, orc):
        out, lse = self.run(self.kv4)
        ro, rl = self.oracle(orc)
        assert_close(out, lse, ro, rl, 1.25 if self.gq is not None else 1.0)
        return out, lse


@pytest.mark.parametrize("d,R", [(512, 64), (512, 32), (512, 0), (128, 32), (128, 0)])
@pytest.mark.parametrize("k", [0, 40])
def test_against_the_oracle(orc, d, R, k):
    """Lengths around tile edges, one sequence with a partial first block."""
    Case(4, d, 128 if d == 512 else 16, R, 128, 4, [2, 255, 259, 700], 180, k=k, gains=R > 0).check(orc)


@pytest.mark.parametrize("H", [1, 63, 64, 65, 128])
def test_heads(orc, H):
    Case(2, 512, H, 64, 100, 4, [3, 1000], 251, k=70, seed=H).check(orc)


@pytest.mark.parametrize("W", [0, 1, 64, 200])
def test_windows(orc, W):
    """Also a row with nothing to attend (W = 0, no complete block): zeros."""
    out, lse = Case(3, 128, 5, 32, W, 4, [1, 3, 90], 25, seed=W).check(orc)
    if W == 0:
        assert (out[0] == 0).all()


def test_one_entry_capacity(orc):
    Case(1, 512, 8, 64, 16, 4, [5], 1).check(orc)
    Case(1, 512, 8, 64, 16, 4, [5], 1, k=1).check(orc)


def test_many_splits_and_the_largest_selection(orc):
    Case(2, 512, 128, 64, 128, 4, [40000, 39000], 10001, k=2048).check(orc)
    Case(2, 512, 128, 64, 128, 4, [40000, 9000], 10001).check(orc)
    Case(9, 512, 64, 64, 128, 128, [70000 + i for i in range(9)], 600).check(orc)
    Case(80, 512, 64, 64, 128, 4, [900 + i for i in range(80)], 300, k=64).check(orc)  # one split


def test_window_tiles_spread_over_full_splits(orc):
    """Calls whose tiles fill every split alike (on 148 multiprocessors), with
    one, two and five window tiles, ragged lengths among the rows."""
    Case(8, 512, 128, 64, 128, 4, [4404 - i for i in range(8)], 1100, k=1024).check(orc)
    Case(8, 512, 128, 64, 320, 4, [3327 - 40 * i for i in range(8)], 832, gains=True).check(orc)
    Case(9, 128, 16, 32, 128, 4, [7679 - 500 * i for i in range(9)], 1920).check(orc)
    Case(148, 512, 3, 64, 64, 4, [255 + i for i in range(148)], 100, k=64).check(orc)  # one split


@pytest.mark.parametrize("k", [0, 100])
def test_large_and_small_scales(orc, k):
    """Entries whose scale bytes exceed 128 (values above 12), and entries well
    below one (2^-12): both inside the exact range of fp16."""
    c = Case(2, 512, 20, 64, 128, 4, [900, 800], 230, k=k, scale=40.0)
    assert int(c.kv4[..., 256:272].max()) > 128
    # Logits reach 40 times the usual ones: the weights' error grows with the
    # logits' (each moves by up to 2^-11 of itself).
    out, lse = c.run(c.kv4)
    ro, _ = c.oracle(orc)
    assert attention_errors(out.double().cpu().numpy(), ro)[1] <= 40 * 2.0 ** -11
    Case(2, 512, 20, 64, 128, 4, [900, 800], 230, k=k, scale=2.0 ** -12).check(orc)


@pytest.mark.parametrize("k", [0, 64])
def test_many_small_weights_beside_a_large_one(k):
    """63 entries with weights of 2^-25.2 of the row's largest: together they are
    all of the output's dims 32 .. (the largest weight's entry is zero there).

    qhat is about sqrt(128) in dim 0, so a logit is the entry's dim 0.  Each weight is
    off by at most 2^-29 of the largest and by its logits' rounding (17.5 times
    2^-11), the sum by the output's 2^-8."""
    B = torch.cuda.get_device_properties(0).multi_processor_count  # one split per row
    N = 64
    p = binding.make_params(B, 128, H=2, k=k, window=0, rope_dim=0, m=4)
    rows = torch.zeros(B, N, 128, dtype=torch.bfloat16, device=DEV)
    rows[:, :, 0] = -1.5
    rows[:, :, 32:] = 1.0
    rows[:, 7] = 0.0
    rows[:, 7, 0] = 16.0
    kv4 = binding.mxfp4_cache(p, N)
    binding.mxfp4_cache_write(p, rows, kv4)
    q = torch.zeros(B, 2, 128, dtype=torch.bfloat16, device=DEV)
    q[:, :, 0] = 1.0
    pos = torch.full((B,), 4 * N - 1, dtype=torch.int64, device=DEV)
    kv_tok = torch.zeros(B, 4 * N, 128, dtype=torch.bfloat16, device=DEV)
    sink = torch.full((2,), float("-inf"), device=DEV)
    out = torch.full((B, 2, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = binding.workspace(p, binding.OP_SPARSE_MQA if k else binding.OP_DENSE_MQA, 1, N)
    if k:
        sel = torch.arange(N, dtype=torch.int32, device=DEV).repeat(B, 1)
        cnt = torch.full((B,), N, dtype=torch.int32, device=DEV)
        binding.sparse_mqa_decode_mxfp4(p, q, pos, kv4, sel, cnt, kv_tok, sink, out, ws=ws)
    else:
        binding.dense_mqa_decode_mxfp4(p, q, pos, kv4, kv_tok, sink, out, ws=ws)
    small = np.exp(-17.5 / np.sqrt(1 + 128 * p.eps))
    want = 63 * small / (1 + 63 * small)
    tol = want * (2.0 ** -29 / small + 17.5 * 2.0 ** -11 + 2.0 ** -8)
    got = out[:, :, 32:].double()
    assert (got - want).abs().max().item() <= tol
    assert (out[:, :, 0].double() - 16).abs().max().item() <= 16 * 2.0 ** -8


@pytest.mark.parametrize("k", [0, 100])
def test_scales_outside_fp16(orc, k):
    """Scale bytes above 140 (values above 49152) are reported and make their
    rows infinite or NaN; scales below 2^-24 count as zeros."""
    c = Case(2, 512, 20, 64, 0, 4, [900, 800], 230, k=k)
    e = int(c.sel[1, 3]) if k else 3
    c.kv4[1, e, 256 + 5] = 141
    out, _ = c.run(c.kv4, status=2)
    bad = ~torch.isfinite(out.float())
    assert bad[1].any(-1).all() and not bad[0].any()
    c.kv4[1, e, 256 + 5] = 140
    out, _ = c.run(c.kv4)
    assert torch.isfinite(out.float()).all()
    c = Case(2, 512, 20, 64, 128, 4, [900, 800], 230, k=k, scale=1e-30)
    out, lse = c.run(c.kv4)
    ro, rl = c.oracle(orc)
    assert_close(out, lse, ro, rl)


def test_entry_offset(orc):
    """A cache that starts at entry 100 of its sequence: as the whole cache."""
    for k in (0, 60):
        c = Case(2, 512, 16, 64, 0, 4, [4 * 300 + 2, 4 * 120], 150, k=k, offset=100)
        out, lse = c.run(c.kv4)
        w = Case(2, 512, 16, 64, 0, 4, [4 * 300 + 2, 4 * 120], 250, k=k)
        w.kv4[:, 100:] = c.kv4
        w.q, w.sink = c.q, c.sink
        if k:
            w.sel = torch.where(c.sel >= 0, c.sel + 100, c.sel)
            w.cnt = c.cnt
            out2, lse2 = w.run(w.kv4)
        else:  # entries 100 .. only: select them
            n = max((4 * 300 + 3) // 4 - 100, 0)
            w.k = n = min(n, 150)
            w.p.k = n
            w.sel = (torch.arange(n, device=DEV, dtype=torch.int32) + 100).repeat(2, 1).contiguous()
            w.cnt = torch.tensor([n, (4 * 120 + 1) // 4 - 100], dtype=torch.int32, device=DEV)
            out2, lse2 = w.run(w.kv4)
        assert_close(out, lse, out2.double().cpu().numpy(), f32(lse2).astype(np.float64))


def test_unselected_and_invisible_entries_are_never_read():
    """NaN entries that no row selects, or that lie past the visible ones,
    change nothing; a selected one makes its rows NaN."""
    c = Case(2, 512, 16, 64, 128, 4, [500, 700], 400, k=50)
    ref = c.run(c.kv4)
    keep = torch.zeros(2, 400, dtype=torch.bool, device=DEV)
    for b in range(2):
        keep[b, c.sel[b].long()] = True
    poisoned = c.kv4.clone()
    poisoned[~keep] = 255
    got = c.run(poisoned)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    poisoned[1, c.sel[1, 7].long()] = 255
    got = c.run(poisoned)
    assert torch.equal(ref[0][0], got[0][0]) and torch.isnan(got[0][1].float()).all()
    d = Case(2, 512, 16, 64, 128, 4, [500, 702], 400)
    ref = d.run(d.kv4)
    poisoned = d.kv4.clone()
    poisoned[0, 125:] = 255
    poisoned[1, 175:] = 255
    got = d.run(poisoned)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])


def test_bad_indices_and_counts(orc):
    """Indices past the visible entries or below -1 are reported and skipped;
    counts outside 0..k are clamped."""
    c = Case(3, 512, 16, 64, 128, 4, [500, 700, 600], 400, k=50)
    good = c.sel.clone(), c.cnt.clone()
    c.sel[0, 3], c.sel[1, 49], c.sel[2, 0] = 125, -5, 1 << 30
    out, lse = c.run(c.kv4, status=7)
    c.cnt -= 1
    for b, j in ((0, 3), (1, 49), (2, 0)):
        row = good[0][b].tolist()
        c.sel[b, :49] = torch.tensor(row[:j] + row[j + 1:], dtype=torch.int32)
    ro, rl = c.oracle(orc)
    assert_close(out, lse, ro, rl)
    c = Case(3, 512, 16, 64, 128, 4, [500, 700, 600], 400, k=50)
    c.cnt[0], c.cnt[1], c.cnt[2] = -3, 0, 999
    out, lse = c.run(c.kv4)
    c.cnt[0], c.cnt[2] = 0, 50
    ro, rl = c.oracle(orc)
    assert_close(out, lse, ro, rl)


def test_repeated_index_counts_twice(orc):
    c = Case(1, 128, 8, 32, 32, 4, [600], 150, k=30)
    c.sel[0, 10:20] = c.sel[0, 10]
    c.check(orc)


def test_entries_past_four_gigabytes():
    """A cache longer than 2^32 bytes: entries at its end, written, read back and
    attended to, as in a short cache."""
    d, N, n = 512, 16_000_000, 96
    short = Case(1, d, 16, 64, 0, 1, [n - 1], n, k=n, seed=7)
    p = binding.make_params(1, d, H=16, k=n, window=0, rope_dim=64, m=1)
    kv4 = binding.mxfp4_cache(p, N)
    assert kv4.numel() > 2 ** 32
    rows = short.values()
    first = torch.tensor([N - n], device=DEV)
    binding.mxfp4_cache_write(p, rows, kv4, first_entry=first)
    # (Not the short cache's bytes: a block whose largest stored value is 3 * 2^e
    # fits the scale 2^(e-1) exactly, so quantising it again halves the scale.)
    assert np.array_equal(kv4[0, N - n:].cpu().numpy(), mxref.cache_rows(mxref.bf16_values(rows[0])))
    back = torch.empty_like(rows)
    binding.mxfp4_cache_read(p, kv4, back, idx=(N - n + torch.arange(
        n, device=DEV, dtype=torch.int32)).view(1, n))
    assert torch.equal(back, rows)
    # (Without rotation, since the query's goes by its position.)
    p0 = binding.make_params(1, d, H=16, k=n, window=0, rope_dim=0, m=1)
    ws = binding.workspace(p0, binding.OP_SPARSE_MQA, 1, N)
    outs = []
    for cache, pos, sel in ((short.kv4, n - 1, torch.arange(n)), (kv4, N - 1,
                                                                  N - n + torch.arange(n))):
        out = torch.empty(1, 16, d, dtype=torch.bfloat16, device=DEV)
        binding.sparse_mqa_decode_mxfp4(p0, short.q, torch.tensor([pos], device=DEV), cache,
                                        sel.int().view(1, n).to(DEV),
                                        torch.tensor([n], dtype=torch.int32, device=DEV),
                                        short.kv_tok, short.sink, out, ws=ws)
        outs.append(out)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])


def test_two_streams_two_workspaces():
    """Two calls at once, each with its own workspace, repeat each other."""
    a = Case(2, 512, 128, 64, 128, 4, [9000, 7000], 2300, k=512, seed=3)
    b = Case(2, 512, 128, 64, 128, 4, [9000, 7000], 2300, seed=4)
    ra, rb = a.run(a.kv4)[0], b.run(b.kv4)[0]
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    wa = binding.workspace(a.p, binding.OP_SPARSE_MQA, 1, 2300)
    wb = binding.workspace(b.p, binding.OP_DENSE_MQA, 1, 2300)
    oa, ob = torch.empty_like(ra), torch.empty_like(rb)
    torch.cuda.synchronize()
    for _ in range(5):
        binding.sparse_mqa_decode_mxfp4(a.p, a.q, a.pos, a.kv4, a.sel, a.cnt, a.kv_tok, a.sink, oa,
                                        ws=wa, stream=sa)
        binding.dense_mqa_decode_mxfp4(b.p, b.q, b.pos, b.kv4, b.kv_tok, b.sink, ob, ws=wb,
                                       stream=sb)
    torch.cuda.synchronize()
    assert torch.equal(oa, ra) and torch.equal(ob, rb)


@pytest.mark.parametrize("k", [0, 128])
def test_back_to_back_calls_behind_other_work(k):
    """Calls that follow copies and one another (each may be scheduled while the
    one before still runs), eager and captured: the same outputs every time."""
    c = Case(8, 512, 128, 64, 128, 4, [4000 - 100 * i for i in range(8)], 1024, k=k, seed=9)
    op = binding.OP_SPARSE_MQA if k else binding.OP_DENSE_MQA
    ws = binding.workspace(c.p, op, 1, 1024)
    qs = [c.q, -c.q, c.q.roll(1, 0)]
    want = []
    for q in qs:
        c.q = q
        want.append(c.run(c.kv4)[0])
    q, cache = torch.empty_like(qs[0]), torch.empty_like(c.kv4)
    outs = [torch.empty_like(w) for w in want]

    def chain():
        cache.copy_(c.kv4)
        for x, out in zip(qs, outs):
            q.copy_(x)
            if k:
                binding.sparse_mqa_decode_mxfp4(c.p, q, c.pos, cache, c.sel, c.cnt, c.kv_tok,
                                                c.sink, out, ws=ws)
            else:
                binding.dense_mqa_decode_mxfp4(c.p, q, c.pos, cache, c.kv_tok, c.sink, out, ws=ws)
        cache.zero_()

    def check():
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
        for o in outs:
            o.zero_()

    for _ in range(10):
        chain()
        check()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        chain()
    for _ in range(10):
        g.replay()
        check()


def _step_inputs(w, L_cap):
    kv_tok, idx_tok = synth.token_streams(w, L_cap=L_cap, device=DEV)
    return kv_tok, idx_tok, synth.pool_params(w, DEV), (
        synth.pool_params(w, DEV, indexer=True) if w.csa else None)


def test_csa_decode_loop(orc):
    """Write, index, select and attend, step by step: prompt compressed into the
    4-bit cache, then six steps across block boundaries, captured into a graph
    at the third.  The newest entry's bytes are those of the bf16 entry; the
    attention is checked against the oracle on the stored values."""
    w = configs.scaled(configs.CSA_128K, B=3, k=64, L=2048)
    B, m, L_cap, N = 3, 4, 2048, 512
    start = np.array([301, 514, 127])
    kv_tok, idx_tok, (w_s, b_pos), (w_si, b_pi) = _step_inputs(w, L_cap)
    p = binding.params_for(w, B=B)
    kv4 = binding.mxfp4_cache(p, N)
    key = torch.zeros(B, N, w.D_I, dtype=torch.uint8, device=DEV)
    ksc = torch.zeros(B, N, device=DEV)
    ctx = torch.from_numpy(start).to(DEV)
    binding.csa_compress_mxfp4(p, kv_tok, ctx, w_s, b_pos, None, 0, N, kv4, idx_tok, w_si, b_pi, key,
                               ksc)
    kv_c = torch.zeros(B, N, w.d, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    pos = torch.empty(B, dtype=torch.int64, device=DEV)
    qi = synth.queries(w, Q=1, device=DEV)
    q, q_idx, q_sc, wt = (qi[n][:, 0].contiguous() for n in ("q", "q_idx", "q_scale", "w"))
    out = torch.empty(B, w.H, w.D, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(B, w.H, device=DEV)
    tidx = torch.empty(B, w.k, dtype=torch.int32, device=DEV)
    tcnt = torch.empty(B, dtype=torch.int32, device=DEV)
    ws = binding.workspace(p, binding.OP_CSA_DECODE_STEP, 1, N)
    step = binding.CsaDecodeStep(p, kv_tok, idx_tok, w_s, b_pos, None, w_si, b_pi, kv4, key, ksc,
                                 qi["sink"], tidx, tcnt, ws, dev_status=st)
    graph = None
    for n in range(6):
        pos.copy_(torch.from_numpy(start + n))
        if n < 2:
            binding.csa_decode_step_mxfp4(p, pos, kv_tok, idx_tok, w_s, b_pos, None, w_si, b_pi, kv4,
                                          key, ksc, q, q_idx, q_sc, wt, qi["sink"], tidx, tcnt, out,
                                          lse=lse, ws=ws, dev_status=st)
        elif n == 2:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                step(pos, q, q_idx, q_sc, wt, out, lse)
        if graph is not None:
            graph.replay()
        torch.cuda.synchronize()
        assert st.item() == 0
        at = (start + n) // m
        for b in range(B):
            binding.csa_compress(p, kv_tok, pos + 1, w_s, b_pos, None, int(at[b]), 1, kv_c)
        stored = kv4.cpu().numpy()
        for b in range(B):
            ref = mxref.cache_rows(mxref.bf16_values(kv_c[b, at[b]]))
            assert np.array_equal(stored[b, at[b]], ref), (n, b)
        vals = torch.empty_like(kv_c)
        binding.mxfp4_cache_read(p, kv4, vals)
        ro, rl = orc.mqa(bits16(q).reshape(B, 1, w.H, w.D), (start + n).reshape(B, 1), bits16(vals),
                         bits16(kv_tok), f32(qi["sink"]), m, w.W, w.rope_dim,
                         tidx.cpu().numpy()[:, None], tcnt.cpu().numpy()[:, None])
        assert_close(out, lse, ro[:, 0], rl[:, 0])
        assert tcnt.tolist() == [min(64, (x + n + 1) // m) for x in start]


def test_hca_decode_loop(orc):
    w = configs.scaled(configs.HCA_1M, B=2, L=1536)
    B, m, N = 2, 128, 12
    start = np.array([125, 640])
    kv_tok, _, (w_s, b_pos), _ = _step_inputs(w, 1536)
    p = binding.params_for(w, B=B)
    kv4 = binding.mxfp4_cache(p, N)
    binding.hca_compress_mxfp4(p, kv_tok, torch.from_numpy(start).to(DEV), w_s, b_pos, None, 0, N, kv4)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    qi = synth.queries(w, Q=1, device=DEV)
    q = qi["q"][:, 0].contiguous()
    ws = binding.workspace(p, binding.OP_HCA_DECODE_STEP, 1, N)
    step = binding.HcaDecodeStep(p, kv_tok, w_s, b_pos, None, kv4, qi["sink"], ws, dev_status=st)
    for n in range(6):
        pos = torch.from_numpy(start + n).to(DEV)
        out = torch.empty(B, w.H, w.D, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(B, w.H, device=DEV)
        if n % 2:
            step(pos, q, out, lse)
        else:
            binding.hca_decode_step_mxfp4(p, pos, kv_tok, w_s, b_pos, None, kv4, q, qi["sink"], out,
                                          lse=lse, ws=ws, dev_status=st)
        torch.cuda.synchronize()
        assert st.item() == 0
        vals = torch.empty(B, N, w.d, dtype=torch.bfloat16, device=DEV)
        binding.mxfp4_cache_read(p, kv4, vals)
        ro, rl = orc.mqa(bits16(q).reshape(B, 1, w.H, w.D), (start + n).reshape(B, 1), bits16(vals),
                         bits16(kv_tok), f32(qi["sink"]), m, w.W, w.rope_dim)
        assert_close(out, lse, ro[:, 0], rl[:, 0])
    kv_c = torch.zeros(B, N, w.d, dtype=torch.bfloat16, device=DEV)
    binding.hca_compress(p, kv_tok, torch.from_numpy(start + 6).to(DEV), w_s, b_pos, None, 0, N, kv_c)
    for b in range(B):
        n = (start[b] + 5) // m + 1
        assert np.array_equal(kv4[b, :n].cpu().numpy(), mxref.cache_rows(mxref.bf16_values(kv_c[b, :n])))


@pytest.mark.parametrize("P,T", [(0, 1), (0, 70), (256, 37)])
def test_csa_prefill_chunk(orc, P, T):
    w = configs.scaled(configs.CSA_128K, B=1, k=32)
    m, L = 4, P + T
    N = -(-L // m) + 1
    kv_tok, idx_tok, (w_s, b_pos), (w_si, b_pi) = _step_inputs(w, L)
    p = binding.params_for(w, B=1)
    kv4 = binding.mxfp4_cache(p, N)
    key = torch.zeros(1, N, w.D_I, dtype=torch.uint8, device=DEV)
    ksc = torch.zeros(1, N, device=DEV)
    if P:
        binding.csa_compress_mxfp4(p, kv_tok, torch.tensor([P], device=DEV), w_s, b_pos, None, 0,
                                   P // m, kv4, idx_tok, w_si, b_pi, key, ksc)
    qi = synth.queries(w, Q=T, device=DEV)
    out = torch.empty(T, w.H, w.D, dtype=torch.bfloat16, device=DEV)
    tidx = torch.empty(T, w.k, dtype=torch.int32, device=DEV)
    tcnt = torch.empty(T, dtype=torch.int32, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = binding.workspace(p, binding.OP_PREFILL, T, N)
    binding.csa_prefill_chunk_mxfp4(p, P, T, kv_tok, idx_tok, w_s, b_pos, None, w_si, b_pi, kv4, key,
                                    ksc, qi["q"][0], qi["q_idx"][0], qi["q_scale"][0], qi["w"][0],
                                    qi["sink"], tidx, tcnt, out, ws=ws, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    vals = torch.empty(1, N, w.d, dtype=torch.bfloat16, device=DEV)
    binding.mxfp4_cache_read(p, kv4, vals)
    pos = (P + np.arange(T)).reshape(1, T)
    ro, _ = orc.mqa(bits16(qi["q"]), pos, bits16(vals), bits16(kv_tok), f32(qi["sink"]), m, w.W,
                    w.rope_dim, tidx.cpu().numpy()[None], tcnt.cpu().numpy()[None])
    assert_close(out, None, ro[0], None)
    kv_c = torch.zeros(1, N, w.d, dtype=torch.bfloat16, device=DEV)
    binding.csa_compress(p, kv_tok, torch.tensor([L], device=DEV), w_s, b_pos, None, 0, N, kv_c)
    assert np.array_equal(kv4[0, : -(-L // m)].cpu().numpy(),
                          mxref.cache_rows(mxref.bf16_values(kv_c[0, : -(-L // m)])))


@pytest.mark.parametrize("P,T", [(0, 130), (256, 5)])
def test_hca_prefill_chunk(orc, P, T):
    w = configs.scaled(configs.HCA_1M, B=1)
    m, L = 128, P + T
    N = -(-L // m)
    kv_tok, _, (w_s, b_pos), _ = _step_inputs(w, L)
    p = binding.params_for(w, B=1)
    kv4 = binding.mxfp4_cache(p, N)
    if P:
        binding.hca_compress_mxfp4(p, kv_tok, torch.tensor([P], device=DEV), w_s, b_pos, None, 0,
                                   P // m, kv4)
    qi = synth.queries(w, Q=T, device=DEV)
    out = torch.empty(T, w.H, w.D, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(T, w.H, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = binding.workspace(p, binding.OP_HCA_PREFILL, T, N)
    binding.hca_prefill_chunk_mxfp4(p, P, T, kv_tok, w_s, b_pos, None, kv4, qi["q"][0], qi["sink"],
                                    out, lse=lse, ws=ws, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    vals = torch.empty(1, N, w.d, dtype=torch.bfloat16, device=DEV)
    binding.mxfp4_cache_read(p, kv4, vals)
    ro, rl = orc.mqa(bits16(qi["q"]), (P + np.arange(T)).reshape(1, T), bits16(vals), bits16(kv_tok),
                     f32(qi["sink"]), m, w.W, w.rope_dim)
    assert_close(out, lse, ro[0], rl[0])


@pytest.mark.parametrize("k", [0, 100])
@pytest.mark.parametrize("B", [2, 150])  # several splits, one
@pytest.mark.parametrize("byte,status", [(255, 0), (141, 2), (142, 2), (200, 2), (254, 2)])
def test_scales_without_an_fp16_value_make_their_rows_nan(k, B, byte, status):
    """A scale byte of 255 is a NaN block whatever its codes (here 0.5 .. 6 and
    their negatives; the library itself writes zeros), and one above 140 is
    reported; both make the row NaN in every dim, alone in its tile (entry 64
    of 65, no window) or not."""
    for n, e in ((65, 64), (65, 3), (1, 0)):
        c = Case(B, 128, 20, 32, 0, 4, [4 * n - 1] * B, n, k=min(k, n))
        ref = c.run(c.kv4)
        b = B - 1
        for codes in (0x11, 0xF1, 0x00):
            bad = c.kv4.clone()
            bad[b, e, 16:32] = codes
            bad[b, e, 64 + 1] = byte
            out, lse = c.run(bad, status=status)
            assert torch.isnan(out[b].float()).all() and torch.isnan(lse[b]).all()
            assert torch.equal(out[:b], ref[0][:b]) and torch.equal(lse[:b], ref[1][:b])

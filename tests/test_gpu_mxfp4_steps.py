"""GPU tests of the decode steps and prefill chunks on a 4-bit cache against the
same call on a bf16 cache: the same indexer keys and selection, every entry's bytes
those of the bf16 entry, and outputs that the attention over the stored values
gives (the stand-alone attention on the same selection, or the fp64 oracle)."""
import numpy as np
import pytest
import torch

import mxref
from compressed_sparse_kv_04_b200 import binding, configs, synth
from gpuhelp import bits16, f32
from test_gpu_mxfp4_attention import assert_close

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    binding.lib()


def same_entries(kv4, kv_c, b, lo, hi):
    got = kv4[b, lo:hi].cpu().numpy()
    assert np.array_equal(got, mxref.cache_rows(mxref.bf16_values(kv_c[b, lo:hi])))


@pytest.mark.parametrize("name", ["tiny", "128k"])
@pytest.mark.parametrize("overlap,offset,W", [(0, 0, 128), (4, 0, 128), (4, 30, 0), (0, 75, 0)])
def test_csa_step_as_on_a_bf16_cache(name, overlap, offset, W):
    """Three sequences, one of them with its newest entry in the shard's first
    place; overlapping compression; a shard of the cache (entry_offset)."""
    base = configs.TINY_CSA if name == "tiny" else configs.CSA_128K
    w = configs.scaled(base, B=3, k=24, L=1200, overlap=overlap, W=W)
    B, m, N, d = 3, w.m, 250 - offset, w.d
    pos = np.array([4 * 249 + 1, 4 * 120 + 3, 4 * offset + 2])
    kv_tok, idx_tok = synth.token_streams(w, L_cap=1200, device=DEV)
    w_s, b_pos = synth.pool_params(w, DEV)
    w_si, b_pi = synth.pool_params(w, DEV, indexer=True)
    p = binding.params_for(w, B=B, entry_offset=offset)
    qi = synth.queries(w, Q=1, device=DEV)
    q, q_idx, q_sc, wt = (qi[n][:, 0].contiguous() for n in ("q", "q_idx", "q_scale", "w"))
    gk = synth.gains(d, 5, DEV)
    post = torch.from_numpy(pos).to(DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = binding.workspace(p, binding.OP_CSA_DECODE_STEP, 1, N)
    got = {}
    for mx in (False, True):
        cache = (binding.mxfp4_cache(p, N) if mx else
                 torch.zeros(B, N, d, dtype=torch.bfloat16, device=DEV))
        key = torch.zeros(B, N, w.D_I, dtype=torch.uint8, device=DEV)
        ksc = torch.zeros(B, N, device=DEV)
        sfx = "_mxfp4" if mx else ""
        getattr(binding, "csa_compress" + sfx)(p, kv_tok, post, w_s, b_pos, gk, 0, N, cache, idx_tok,
                                               w_si, b_pi, key, ksc)
        out = torch.full((B, w.H, d), float("nan"), dtype=torch.bfloat16, device=DEV)
        lse = torch.full((B, w.H), float("nan"), device=DEV)
        tidx = torch.empty(B, w.k, dtype=torch.int32, device=DEV)
        tcnt = torch.empty(B, dtype=torch.int32, device=DEV)
        getattr(binding, "csa_decode_step" + sfx)(
            p, post, kv_tok, idx_tok, w_s, b_pos, gk, w_si, b_pi, cache, key, ksc, q, q_idx, q_sc, wt,
            qi["sink"], tidx, tcnt, out, gamma_kv=gk, lse=lse, ws=ws, dev_status=st)
        got[mx] = cache, key, ksc, tidx, tcnt, out, lse
    torch.cuda.synchronize()
    assert st.item() == 0
    for i in (1, 2, 3, 4):
        assert torch.equal(got[False][i], got[True][i])
    for b in range(B):
        same_entries(got[True][0], got[False][0], b, 0, int(pos[b] // m) + 1 - offset)
    kv4, _, _, tidx, tcnt, out, lse = got[True]
    assert tcnt.tolist() == [min(24, max(0, (int(x) + 1) // m - offset)) for x in pos]
    ref, rlse = torch.empty_like(out), torch.empty_like(lse)
    binding.sparse_mqa_decode_mxfp4(p, q, post, kv4, tidx, tcnt, kv_tok, qi["sink"], ref,
                                    gamma_kv=gk, lse=rlse,
                                    ws=binding.workspace(p, binding.OP_SPARSE_MQA, 1, N))
    assert_close(out, lse, ref.double().cpu().numpy(), f32(rlse).astype(np.float64), 1.25)


@pytest.mark.parametrize("P,T", [(512, 517), (64, 1203)])
def test_csa_chunk_of_many_queries(orc, P, T):
    w = configs.scaled(configs.CSA_128K, B=1, k=40, H=20)
    m, L = w.m, P + T
    N = -(-L // m)
    kv_tok, idx_tok = synth.token_streams(w, L_cap=L, device=DEV)
    w_s, b_pos = synth.pool_params(w, DEV)
    w_si, b_pi = synth.pool_params(w, DEV, indexer=True)
    p = binding.params_for(w, B=1)
    qi = synth.queries(w, Q=T, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = binding.workspace(p, binding.OP_PREFILL, T, N)
    got = {}
    for mx in (False, True):
        cache = (binding.mxfp4_cache(p, N) if mx else
                 torch.zeros(1, N, w.d, dtype=torch.bfloat16, device=DEV))
        key = torch.zeros(1, N, w.D_I, dtype=torch.uint8, device=DEV)
        ksc = torch.zeros(1, N, device=DEV)
        sfx = "_mxfp4" if mx else ""
        getattr(binding, "csa_compress" + sfx)(p, kv_tok, torch.tensor([P], device=DEV), w_s, b_pos,
                                               None, 0, P // m, cache, idx_tok, w_si, b_pi, key, ksc)
        out = torch.full((T, w.H, w.d), float("nan"), dtype=torch.bfloat16, device=DEV)
        tidx = torch.empty(T, w.k, dtype=torch.int32, device=DEV)
        tcnt = torch.empty(T, dtype=torch.int32, device=DEV)
        getattr(binding, "csa_prefill_chunk" + sfx)(
            p, P, T, kv_tok, idx_tok, w_s, b_pos, None, w_si, b_pi, cache, key, ksc, qi["q"][0],
            qi["q_idx"][0], qi["q_scale"][0], qi["w"][0], qi["sink"], tidx, tcnt, out, ws=ws,
            dev_status=st)
        got[mx] = cache, key, ksc, tidx, tcnt, out
    torch.cuda.synchronize()
    assert st.item() == 0
    for i in (1, 2, 3, 4):
        assert torch.equal(got[False][i], got[True][i])
    same_entries(got[True][0], got[False][0], 0, 0, N)
    kv4, _, _, tidx, tcnt, out = got[True]
    vals = torch.empty(1, N, w.d, dtype=torch.bfloat16, device=DEV)
    binding.mxfp4_cache_read(p, kv4, vals)
    ro, _ = orc.mqa(bits16(qi["q"]), (P + np.arange(T)).reshape(1, T), bits16(vals), bits16(kv_tok),
                    f32(qi["sink"]), m, w.W, w.rope_dim, tidx.cpu().numpy()[None],
                    tcnt.cpu().numpy()[None])
    assert_close(out, None, ro[0], None)


@pytest.mark.parametrize("P,T", [(384, 601), (0, 1100)])
def test_hca_chunk_of_many_queries(orc, P, T):
    w = configs.scaled(configs.HCA_1M, B=1, H=20)
    m, L = w.m, P + T
    N = -(-L // m)
    kv_tok, _ = synth.token_streams(w, L_cap=L, device=DEV)
    w_s, b_pos = synth.pool_params(w, DEV)
    p = binding.params_for(w, B=1)
    qi = synth.queries(w, Q=T, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = binding.workspace(p, binding.OP_HCA_PREFILL, T, N)
    kv4 = binding.mxfp4_cache(p, N)
    if P:
        binding.hca_compress_mxfp4(p, kv_tok, torch.tensor([P], device=DEV), w_s, b_pos, None, 0,
                                   P // m, kv4)
    out = torch.full((T, w.H, w.d), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, w.H), float("nan"), device=DEV)
    binding.hca_prefill_chunk_mxfp4(p, P, T, kv_tok, w_s, b_pos, None, kv4, qi["q"][0], qi["sink"],
                                    out, lse=lse, ws=ws, dev_status=st)
    kv_c = torch.zeros(1, N, w.d, dtype=torch.bfloat16, device=DEV)
    binding.hca_compress(p, kv_tok, torch.tensor([L], device=DEV), w_s, b_pos, None, 0, N, kv_c)
    torch.cuda.synchronize()
    assert st.item() == 0
    same_entries(kv4, kv_c, 0, 0, N)
    vals = torch.empty(1, N, w.d, dtype=torch.bfloat16, device=DEV)
    binding.mxfp4_cache_read(p, kv4, vals)
    ro, rl = orc.mqa(bits16(qi["q"]), (P + np.arange(T)).reshape(1, T), bits16(vals), bits16(kv_tok),
                     f32(qi["sink"]), m, w.W, w.rope_dim)
    assert_close(out, lse, ro[0], rl[0])

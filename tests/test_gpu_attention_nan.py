"""GPU tests of NaN in the attention, over bf16 and over 4-bit caches: a query
head, an attended entry or an attended window token that is NaN makes the rows
it enters NaN (output and log-sum-exp), wherever it falls in the list: alone in
its tile or split, before or after finite tiles, with one split and with
several.  Every other row keeps its bits.

A softmax over a list with a NaN logit has NaN weights, so every dim of the
output is NaN by the formula."""
import pytest
import torch

from compressed_sparse_kv_04_b200 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN = float("nan")
INF = float("inf")
# Rows that fill the multiprocessors (with one and with two head groups), so that
# each takes one split.
ONE_SPLIT = 150


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    binding.lib()


class Case:
    """B rows of H heads over n_vis entries each (all of them selected where
    `sparse`) and a window of W tokens."""

    def __init__(self, mx, sparse, B, n_vis, W=0, H=20, d=128, R=32, sink=None, seed=1):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.mx, self.sparse, self.B, self.n_vis, self.H, self.d = mx, sparse, B, n_vis, H, d
        self.N = max(n_vis, 1)
        self.p = binding.make_params(B, d, H=H, k=n_vis if sparse else 0, window=W, rope_dim=R, m=4)
        L = 4 * self.N + 3
        pos = 4 * n_vis + 2
        self.pos = torch.full((B,), pos, dtype=torch.int64, device=DEV)
        self.bf = torch.randn(B, self.N, d, generator=g, device=DEV).bfloat16()
        self.kv4 = binding.mxfp4_cache(self.p, self.N)
        binding.mxfp4_cache_write(self.p, self.bf, self.kv4)
        self.tok = torch.randn(B, L, d, generator=g, device=DEV).bfloat16()
        self.last = pos
        self.q = torch.randn(B, H, d, generator=g, device=DEV).bfloat16()
        self.sink = torch.randn(H, generator=g, device=DEV) if sink is None else torch.full(
            (H,), sink, device=DEV)
        self.sel = torch.arange(max(n_vis, 1), dtype=torch.int32, device=DEV).repeat(B, 1)
        self.cnt = torch.full((B,), n_vis, dtype=torch.int32, device=DEV)
        op = binding.OP_SPARSE_MQA if sparse else binding.OP_DENSE_MQA
        self.ws = binding.workspace(self.p, op, 1, self.N)

    def poison(self, b, lo, hi=None):
        """Entries lo .. hi - 1 of sequence b: NaN in one block of 32 dims."""
        hi = lo + 1 if hi is None else hi
        if self.mx:
            self.kv4[b, lo:hi, 32:48] = 0
            self.kv4[b, lo:hi, self.d // 2 + 2] = 255
        else:
            self.bf[b, lo:hi, 70] = NAN

    def run(self):
        out = torch.full((self.B, self.H, self.d), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((self.B, self.H), 7.0, device=DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        kw = dict(lse=lse, ws=self.ws, dev_status=st)
        cache = self.kv4 if self.mx else self.bf
        sel = (self.sel, self.cnt) if self.sparse else ()
        name = "sparse_mqa_decode" if self.sparse else "dense_mqa_decode"
        getattr(binding, name + ("_mxfp4" if self.mx else ""))(
            self.p, self.q, self.pos, cache, *sel, self.tok, self.sink, out, **kw)
        torch.cuda.synchronize()
        assert st.item() == 0
        return out.float(), lse

    def clean(self):
        """The finite result, before anything is poisoned."""
        out, lse = self.run()
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        return out, lse

    def check(self, before, rows, heads=None):
        """Rows (and heads) NaN in every dim, the others as before."""
        bad = torch.zeros(self.B, self.H, dtype=torch.bool, device=DEV)
        for b in rows:
            bad[b, slice(None) if heads is None else heads] = True
        out, lse = self.run()
        assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
        assert torch.equal(out[~bad], before[0][~bad]) and torch.equal(lse[~bad], before[1][~bad])


BOTH = pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp4"])
KIND = pytest.mark.parametrize("sparse", [False, True], ids=["dense", "sparse"])


@BOTH
@KIND
@pytest.mark.parametrize("d,R,H", [(128, 32, 20), (512, 64, 70)])
@pytest.mark.parametrize("n_vis", [1, 65, 193])
def test_an_entry_alone_in_its_split(mx, sparse, d, R, H, n_vis):
    """The newest entry, alone in the last tile, which is a split of its own."""
    c = Case(mx, sparse, 2, n_vis, H=H, d=d, R=R)
    before = c.clean()
    c.poison(1, n_vis - 1)
    c.check(before, [1])


@BOTH
@KIND
@pytest.mark.parametrize("d,R,H", [(128, 32, 20), (512, 64, 70)])
@pytest.mark.parametrize("lo,hi,n_vis", [(0, 1, 1), (64, 65, 65), (0, 64, 130), (64, 128, 130),
                                         (128, 130, 130), (0, 130, 130)])
def test_tiles_of_one_split(mx, sparse, d, R, H, lo, hi, n_vis):
    """One split per row: a tile of nothing but NaN before, between and after
    finite tiles, and nothing but NaN."""
    c = Case(mx, sparse, ONE_SPLIT, n_vis, H=H, d=d, R=R)
    before = c.clean()
    c.poison(3, lo, hi)
    c.check(before, [3])


@BOTH
@KIND
@pytest.mark.parametrize("B", [1, ONE_SPLIT])
def test_an_entry_beside_the_window(mx, sparse, B):
    """The only entry is NaN, 70 window tokens are not."""
    c = Case(mx, sparse, B, 1, W=70, d=512, R=64, H=16)
    before = c.clean()
    c.poison(B - 1, 0)
    c.check(before, [B - 1])


@BOTH
@KIND
@pytest.mark.parametrize("B", [1, ONE_SPLIT])
@pytest.mark.parametrize("W", [1, 70])
def test_window_tokens(mx, sparse, B, W):
    """The newest token, alone in the window or last in it."""
    c = Case(mx, sparse, B, 100, W=W, d=512, R=64, H=16)
    before = c.clean()
    c.tok[B - 1, c.last, 9] = NAN
    c.check(before, [B - 1])


@BOTH
@KIND
@pytest.mark.parametrize("B", [3, ONE_SPLIT])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_queries(mx, sparse, B, value):
    """One head's query, and every head of another row."""
    c = Case(mx, sparse, B, 150, W=70, d=512, R=64, H=70)
    before = c.clean()
    q = c.q.clone()
    c.q[1, 66, 5] = value
    c.check(before, [1], heads=66)
    c.q = q
    c.q[2, :, 500] = value
    c.check(before, [2])


@BOTH
@KIND
@pytest.mark.parametrize("B", [3, ONE_SPLIT])
@pytest.mark.parametrize("sink", [-INF, INF])
def test_infinite_sinks(mx, sparse, B, sink):
    """Without a sink (-infinity), and where the sink takes all of the weight
    (+infinity: zeros): NaN all the same."""
    c = Case(mx, sparse, B, 65, d=128, sink=sink)
    before = c.run()
    assert torch.isfinite(before[0]).all() and (sink < 0 or (before[0] == 0).all())
    c.poison(2, 64)
    c.check(before, [2])


@BOTH
@KIND
@pytest.mark.parametrize("B", [3, ONE_SPLIT])
def test_masked_and_absent_rows_stay_out(mx, sparse, B):
    """NaN entries past the visible ones, unselected ones, and NaN tokens
    outside the window change nothing; a row without anything to attend is
    zeros, its log-sum-exp the sink's, whatever its query holds."""
    c = Case(mx, sparse, B, 130, W=70, d=128)
    pos = c.last if sparse else 4 * 120 + 2
    c.pos[:] = pos
    c.cnt[:] = 120
    before = c.clean()
    c.tok[:, : pos - 69] = NAN
    c.tok[:, pos + 1:] = NAN
    c.poison(slice(None), 120, 130)
    c.check(before, [])
    e = Case(mx, sparse, B, 1, W=0, d=128)
    e.pos[:] = 1  # no entry is visible
    e.cnt[:] = 0
    e.q[:] = NAN
    out, lse = e.run()
    assert (out == 0).all() and torch.allclose(lse, e.sink.expand_as(lse), rtol=2.0 ** -22, atol=0)


@BOTH
@KIND
@pytest.mark.parametrize("B", [2, ONE_SPLIT])
@pytest.mark.parametrize("n_vis", [1, 65, 200])
def test_a_nan_sink(mx, sparse, B, n_vis):
    """A NaN sink makes its head NaN where there is something to attend; a row
    with nothing to attend stays zero, its log-sum-exp the sink's, for one split
    and for several."""
    c = Case(mx, sparse, B, n_vis, d=128)
    c.pos[0] = 1  # row 0: no entry is visible
    c.cnt[0] = 0
    before = c.run()
    assert (before[0][0] == 0).all()
    c.sink[5] = NAN
    out, lse = c.run()
    bad = torch.zeros(B, c.H, dtype=torch.bool, device=DEV)
    bad[:, 5] = True
    assert torch.isnan(lse[bad]).all()
    assert (out[0] == 0).all() and torch.isnan(out[1:, 5]).all()
    assert torch.equal(out[~bad], before[0][~bad]) and torch.equal(lse[~bad], before[1][~bad])


def test_a_shard_of_a_split_context():
    """Partials of two shards merged: the one whose only selected entry is NaN
    is not taken for an empty one."""
    B, H, d, n = 1, 20, 512, 70
    c = Case(False, True, B, n, H=H, d=d, R=64)
    parts = torch.zeros(B, 2, H, d, dtype=torch.float16, device=DEV)
    ml = torch.zeros(B, 2, 2, H, device=DEV)

    def run(bad):
        for r, cnt in enumerate((n, 1)):
            cache = c.bf.clone()
            if bad and r == 1:
                cache[0, 0, 3] = NAN
            o, x = torch.zeros(B, 1, H, d, dtype=torch.float16, device=DEV), torch.zeros(
                B, 1, 2, H, device=DEV)
            binding.sparse_mqa_partials(c.p, 1, c.q, c.pos, cache, c.sel,
                                        torch.tensor([cnt], dtype=torch.int32, device=DEV), c.tok,
                                        o, x)
            parts[:, r], ml[:, r] = o[:, 0], x[:, 0]
        out = torch.empty(B, H, d, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(B, H, device=DEV)
        binding.mqa_merge_partials(c.p, 2, parts, ml, c.pos, c.sink, out, lse=lse)
        torch.cuda.synchronize()
        return out, lse

    out, lse = run(False)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    out, lse = run(True)
    assert torch.isnan(out).all() and torch.isnan(lse).all()

"""The serving operators together, as a speculative decoder uses them over a paged cache: pages for the drafted
tokens, norm + rotation + append, tree attention, the accepted rows kept, pages given back; then forks, a window
decode and the decode step on what is left.  Every step is checked against 64-bit formulas on plain lists."""
import math

import pytest
import torch

from attention_testlib import attend, close

pytestmark = pytest.mark.gpu
D, EPS = 128, 1e-6


@pytest.fixture(scope="module")
def H():
    import hash_aware_top_b200 as H

    return H


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    """A paged cache and, per sequence, the rows (64 bits) that it should hold."""

    def __init__(self, H, dtype, B=4, Hq=8, Hkv=2, max_seq=300, bs=16, T=11, seed=0):
        self.H, self.B, self.Hq, self.Hkv, self.bs, self.T, self.dtype = H, B, Hq, Hkv, bs, T, dtype
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.d = H.dims_for(B, Hq, Hkv, D, 128, max_seq, dtype)
        n = B * (-(-max_seq // bs)) + 3
        self.K, self.V = (torch.full((n, Hkv, bs, D), float("nan"), device="cuda", dtype=dtype) for _ in range(2))
        self.codes = torch.zeros((n, Hkv, bs, 4), dtype=torch.int32, device="cuda")
        self.table = torch.full((B, -(-max_seq // bs)), -1, dtype=torch.int32, device="cuda")
        self.lens, self.ref = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
        self.rope = H.hata_rope_table(max_seq, 128, 10000.0)
        self.wq, self.wk = (1 + 0.2 * torch.randn(D, generator=self.g, device="cuda") for _ in range(2))
        z = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.pages_ws, self.span_ws = z(H.hata_pages_workspace_size(self.d)), z(H.hata_span_workspace_size(self.d, T))
        self.status_ws = z(16)
        self.rows = [[] for _ in range(B)]  # per sequence: (k [Hkv][D], v [Hkv][D]) in 64 bits

    def resize(self, lens):
        self.H.hata_pages_resize(self.d, lens, self.K, self.V, self.codes, self.table, self.bs, self.lens, self.ref, self.pages_ws)

    def append(self, x, n_new, positions, q_out):
        Hq, Hkv = self.Hq, self.Hkv
        self.H.hata_norm_rope_paged(self.d, x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], self.wq, self.wk, EPS, self.rope,
                                    False, n_new, positions, self.lens, q_out, self.K, self.V, self.table, self.bs, self.status_ws)

    def turned(self, x, w, pos):
        """x [H][D] at position pos: normed and rotated, in 64 bits."""
        y = x.double()
        y = y / (y.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w.double()
        c, s = self.rope[pos].double()
        a, b = y[:, :64], y[:, 64:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    def cached(self, b, L):
        at = torch.arange(L, device="cuda")
        page = self.table[b].long()[at // self.bs]
        return self.K[page, :, at % self.bs].transpose(0, 1), self.V[page, :, at % self.bs].transpose(0, 1)

    def check_rows(self):
        """Every row that the sequences hold: keys to the rounding of the type (and fp32 arithmetic, 80 half steps of values
        that a rotation adds up from two), values exactly."""
        assert self.lens.tolist() == [len(r) for r in self.rows]
        half = torch.finfo(self.dtype).eps / 2
        for b, rows in enumerate(self.rows):
            if rows:
                K, V = self.cached(b, len(rows))
                k, v = torch.stack([r[0] for r in rows], 1), torch.stack([r[1] for r in rows], 1)
                tol = half * 1.01 * k.abs() + 80 * 2.0 ** -24 * 2 * k.abs().amax(-1, keepdim=True)
                assert bool(((K.double() - k).abs() <= tol).all()) and torch.equal(V.double(), v)
        for ws in (self.pages_ws, self.span_ws, self.status_ws):
            assert self.H.hata_read_device_status(ws) == 0


def trees(T, B, seed):
    """Parents (an earlier node or -1), the mask words and the depths."""
    r = torch.Generator().manual_seed(seed)
    parent = [[int(torch.randint(-1, i, (1,), generator=r)) if i else -1 for i in range(T)] for _ in range(B)]
    sees = torch.zeros(B, T, T, dtype=torch.bool)
    for b in range(B):
        for i in range(T):
            j = i
            while j >= 0:
                sees[b, i, j] = True
                j = parent[b][j]
    words = torch.zeros(B, T, -(-T // 32) * 32, dtype=torch.int64)
    words[:, :, :T] = sees
    words = (words.view(B, T, -1, 32) << torch.arange(32)).sum(-1)
    return parent, torch.where(words >= 2**31, words - 2**32, words).int().cuda(), sees.cuda(), (sees.sum(-1) - 1).int().cuda()


def draft_round(s, seed):
    """One round for all sequences; returns what was accepted."""
    H, B, T, Hq, Hkv = s.H, s.B, s.T, s.Hq, s.Hkv
    parent, mask, sees, depth = trees(T, B, seed)
    before = s.lens.clone()
    x = torch.randn(B, T, Hq + 2 * Hkv, D, generator=s.g, device="cuda").to(s.dtype)
    q, out = (torch.zeros(B, Hq, T, D, device="cuda", dtype=s.dtype) for _ in range(2))
    s.resize(before + T)
    s.append(x, None, (before[:, None] + depth).int().contiguous(), q)
    H.hata_tree_attention_paged(s.d, q, s.K, s.V, s.table, s.bs, s.lens, None, mask, 0.0, out, s.span_ws)
    keep, n_keep = torch.zeros(B, T, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        path, j = [], (seed * 7 + b * 3) % T
        while j >= 0:
            path.insert(0, j)
            j = parent[b][j]
        keep[b, :len(path)], n_keep[b] = torch.tensor(path), len(path)
    ctx = before.tolist()
    for b in range(B):  # the attention, from what the cache holds
        K, V = s.cached(b, ctx[b] + T)
        vis = torch.ones(T, ctx[b] + T, dtype=torch.bool, device="cuda")
        vis[:, ctx[b]:] = sees[b]
        for h in range(Hq):
            pos = [ctx[b] + int(depth[b, i]) for i in range(T)]
            want_q = torch.stack([s.turned(x[b, i, :Hq], s.wq, pos[i])[h] for i in range(T)])
            half = torch.finfo(s.dtype).eps / 2
            assert bool(((q[b, h].double() - want_q).abs() <= half * 1.01 * want_q.abs() + 80 * 2.0 ** -24 * 2 * want_q.abs().amax()).all())
            want, absv, qk = attend(q[b, h], K[h // (Hq // Hkv)], V[h // (Hq // Hkv)], vis)
            close(out[b, h], want, absv, qk, ctx[b] + T, s.dtype)
        for j in keep[b, : int(n_keep[b])].tolist():
            s.rows[b].append((s.turned(x[b, j, Hq:Hq + Hkv], s.wk, ctx[b] + int(depth[b, j])), x[b, j, Hq + Hkv:].double()))
    new_lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    H.hata_compact_kv_paged(s.d, keep.cuda(), n_keep.cuda(), None, s.lens, s.K, s.V, s.codes, s.table, s.bs, new_lens, s.status_ws)
    s.resize(new_lens)
    s.check_rows()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_speculative_rounds_forks_and_decodes(H, dtype):
    s = Server(H, dtype)
    B, Hq, Hkv = s.B, s.Hq, s.Hkv
    # prompts of different lengths, one of them empty
    n = [37, 0, 16, 90]
    x = torch.randn(B, 90, Hq + 2 * Hkv, D, generator=s.g, device="cuda").to(dtype)
    q = torch.zeros(B, Hq, 90, D, device="cuda", dtype=dtype)
    s.resize(i32(n))
    s.append(x, i32(n), None, q)
    for b in range(B):
        for t in range(n[b]):
            s.rows[b].append((s.turned(x[b, t, Hq:Hq + Hkv], s.wk, t), x[b, t, Hq + Hkv:].double()))
    s.check_rows()
    for seed in range(3):
        draft_round(s, seed)
    # sequence 3 goes on from sequence 0, 1 from 2; then each goes its own way
    H.hata_pages_fork(s.d, i32([0, 2, 2, 0]), s.table, s.bs, s.lens, s.ref, s.pages_ws)
    s.rows[3], s.rows[1] = list(s.rows[0]), list(s.rows[2])
    s.check_rows()
    for seed in range(3, 5):
        draft_round(s, seed)
    # a window decode and the decode step (all rows selected) on the newest token
    lens = [len(r) for r in s.rows]
    qd, out = torch.randn(B, Hq, D, generator=s.g, device="cuda").to(dtype), torch.zeros(B, Hq, D, device="cuda", dtype=dtype)
    H.hata_window_decode_paged(s.d, qd, s.K, s.V, s.table, s.bs, s.lens, 20, 3, 0.0, out, s.span_ws)
    for b in range(B):
        at = torch.arange(lens[b], device="cuda")
        K, V = s.cached(b, lens[b])
        for h in range(Hq):
            want, absv, qk = attend(qd[b, h][None], K[h // 4], V[h // 4], ((at < 3) | (at >= lens[b] - 20))[None])
            close(out[b, h][None], want, absv, qk, 23, dtype)
    W = torch.randn(Hkv, D, 128, generator=s.g, device="cuda") / math.sqrt(D)
    pool = H.dims_for(s.K.shape[0], Hkv, Hkv, D, 128, s.bs, dtype)
    H.hata_encode_append(pool, s.K, Hkv, s.bs, s.bs, None, W, s.codes, s.bs, s.status_ws)
    k = max(lens)
    ws = torch.zeros(H.hata_workspace_size(s.d, k), dtype=torch.uint8, device="cuda")
    out2 = torch.zeros_like(out)
    H.hata_decode_step_paged(s.d, qd, s.K, s.V, W, W, s.codes, s.table, s.bs, s.lens, k, 0.0, out2, None, None, ws)
    assert H.hata_read_device_status(ws) == 0
    for b in range(B):
        K, V = s.cached(b, lens[b])
        for h in range(Hq):
            want, _, _ = attend(qd[b, h][None], K[h // 4], V[h // 4], torch.ones(1, lens[b], dtype=torch.bool, device="cuda"))
            assert float((out2[b, h].double() - want[0]).abs().max()) <= (2e-2 if dtype == torch.bfloat16 else 1e-4)
    s.resize(i32([0] * B))
    assert int(s.ref.abs().sum()) == 0


def test_a_round_captured_and_replayed(H):
    """The whole round in one CUDA graph, replayed on other inputs and lengths, against the same calls made one by one."""
    s = Server(H, torch.bfloat16, T=5)
    B, T, Hq, Hkv = s.B, s.T, s.Hq, s.Hkv
    x = torch.zeros(B, T, Hq + 2 * Hkv, D, device="cuda", dtype=torch.bfloat16)
    q, out = torch.zeros(B, Hq, T, D, device="cuda", dtype=torch.bfloat16), torch.zeros(B, Hq, T, D, device="cuda", dtype=torch.bfloat16)
    start, grown, kept = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
    keep, n_keep = torch.zeros(B, T, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    _, mask, _, _ = trees(T, B, 1)

    def one_round():
        s.resize(start)
        grown.copy_(start + T)
        s.resize(grown)
        s.append(x, None, None, q)
        H.hata_tree_attention_paged(s.d, q, s.K, s.V, s.table, s.bs, s.lens, None, mask, 0.0, out, s.span_ws)
        H.hata_compact_kv_paged(s.d, keep, n_keep, None, s.lens, s.K, s.V, s.codes, s.table, s.bs, kept, s.status_ws)
        s.resize(kept)

    def state():
        return [t.clone() for t in (s.K, s.V, s.codes, s.table, s.lens, s.ref, q, out)]

    def restore(old):
        for t, o in zip((s.K, s.V, s.codes, s.table, s.lens, s.ref, q, out), old):
            t.copy_(o)

    s.K.zero_(), s.V.zero_()
    one_round()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        one_round()
    for seed in range(3):
        x.copy_(torch.randn(x.shape, generator=s.g, device="cuda"))
        start.copy_(i32([40 + seed, 0, 16, 200 - 31 * seed]))
        keep.copy_(i32([[0, 2, 4, 0, 0], [1, 0, 0, 0, 0], [0, 1, 2, 3, 4], [3, 4, 0, 0, 0]]))
        n_keep.copy_(i32([3, 1, 5, 2 - seed % 2]))
        old = state()
        one_round()
        want = state()
        restore(old)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(state(), want):
            assert torch.equal(a, b)
    for ws in (s.pages_ws, s.span_ws, s.status_ws):
        assert H.hata_read_device_status(ws) == 0


def test_two_streams_at_once(H):
    """Tree attention of two caches on two streams, each with its own workspace, gives what each gives alone."""
    def make(seed, Hq):
        g = torch.Generator(device="cuda").manual_seed(seed)
        d = H.dims_for(2, Hq, 2, D, 128, 3000, "bf16")
        r = lambda *n: torch.randn(*n, generator=g, device="cuda").bfloat16()  # noqa: E731
        q, K, V = r(2, Hq, 30, D), r(2, 2, 3000, D), r(2, 2, 3000, D)
        ws = torch.zeros(H.hata_span_workspace_size(d, 30), dtype=torch.uint8, device="cuda")
        return d, q, K, V, i32([3000, 1700]), ws

    cases = [make(1, 8), make(2, 2)]  # the many-row kernel and the few-row kernel
    alone = []
    for d, q, K, V, lens, ws in cases:
        out = torch.zeros_like(q)
        H.hata_tree_attention(d, q, K, V, lens, None, None, 0.0, out, ws)
        alone.append(out)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [torch.zeros_like(c[1]) for c in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, (d, q, K, V, lens, ws), out in zip(streams, cases, outs):
            H.hata_tree_attention(d, q, K, V, lens, None, None, 0.0, out, ws, stream=st)
    torch.cuda.synchronize()
    for a, b in zip(alone, outs):
        assert torch.equal(a, b)

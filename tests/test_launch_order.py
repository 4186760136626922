"""What comes next on a stream after an attention call whose units need no joining finds the call finished: a copy of its
outputs, page bookkeeping that changes the lengths and the table it reads, an append over rows it reads, and the next call on
the same workspace.  A captured sequence of such calls, replayed, gives bit for bit what the calls give one by one with a
synchronisation after each."""
import pytest
import torch

pytestmark = pytest.mark.gpu
D, BS = 128, 64


@pytest.fixture(scope="module")
def H():
    import hash_aware_top_b200 as H

    return H


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Calls:
    """B sequences over a paged cache, their pages allocated by the library."""

    def __init__(self, H, dtype, B, Hq, Hkv, max_seq, T, seed=0):
        self.H, self.dtype, self.B, self.Hq, self.Hkv, self.T = H, dtype, B, Hq, Hkv, T
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.d = H.dims_for(B, Hq, Hkv, D, 128, max_seq, dtype)
        blocks = -(-max_seq // BS)
        n = B * blocks + 5
        r = lambda *s: torch.randn(*s, generator=self.g, device="cuda").to(dtype)  # noqa: E731
        self.K, self.V = r(n, Hkv, BS, D), r(n, Hkv, BS, D)
        self.table = torch.full((B, blocks), -1, dtype=torch.int32, device="cuda")
        self.lens, self.ref = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
        self.q, self.qt = r(B, Hq, D), r(B, Hq, T, D)
        self.x = r(B, T, Hq + 2 * Hkv, D)
        self.out, self.seen, self.out2 = (torch.zeros_like(self.q) for _ in range(3))
        self.tout, self.tseen, self.q_out = (torch.zeros_like(self.qt) for _ in range(3))
        self.n_new, self.none = i32([T] * B), i32([0] * B)
        self.long, self.short = i32([0] * B), i32([0] * B)
        z = lambda k: torch.zeros(k, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.ws = z(max(H.hata_span_workspace_size(self.d, k) for k in (1, T)))
        self.pages_ws, self.status_ws = z(H.hata_pages_workspace_size(self.d)), z(16)

    def resize(self, lens):
        self.H.hata_pages_resize(self.d, lens, self.K, self.V, None, self.table, BS, self.lens, self.ref, self.pages_ws)

    def window(self, out, window=100000):
        self.H.hata_window_decode_paged(self.d, self.q, self.K, self.V, self.table, BS, self.lens, window, 3, 0.0, out, self.ws)

    def tree(self, n_new, out):
        self.H.hata_tree_attention_paged(self.d, self.qt, self.K, self.V, self.table, BS, self.lens, n_new, None, 0.0, out, self.ws)

    def append(self):
        Hq, Hkv, x = self.Hq, self.Hkv, self.x
        self.H.hata_norm_rope_paged(self.d, x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], None, None, 1e-6, None, False,
                                    self.n_new, None, self.lens, self.q_out, self.K, self.V, self.table, BS, self.status_ws)

    def steps(self):
        return [
            lambda: self.resize(self.long),
            lambda: self.window(self.out),
            lambda: self.seen.copy_(self.out),         # an attention output read by the next kernel
            lambda: self.window(self.out2, 77),
            lambda: self.resize(self.short),           # pages and lengths taken away from under a finished call
            lambda: self.resize(self.long),
            lambda: self.tree(self.n_new, self.tout),
            lambda: self.append(),                     # the rows that the tree read
            lambda: self.tree(self.none, self.tout),   # nothing to attend to: the kernels only come and go
            lambda: self.resize(self.short),
            lambda: self.tree(self.n_new, self.tseen),
            lambda: self.window(self.out2, 50),        # the same workspace
            lambda: self.resize(self.none),
        ]

    def state(self):
        return [self.K, self.V, self.table, self.lens, self.ref, self.out, self.seen, self.out2, self.tout, self.tseen, self.q_out]


# units of 128 slots or less, and as many units as let every one run in one CTA; rows of the few-row and of the many-row kernel
@pytest.mark.parametrize("dtype,B,Hq,Hkv,T,max_seq,lens", [
    (torch.bfloat16, 16, 32, 8, 3, 2100, (1900, 2048)), (torch.float32, 16, 16, 8, 2, 2100, (1900, 2048)),
    (torch.bfloat16, 2, 8, 2, 5, 300, (20, 128)), (torch.float32, 3, 4, 4, 4, 300, (20, 128)),
    (torch.bfloat16, 16, 32, 8, 20, 2100, (1900, 2048)), (torch.bfloat16, 2, 8, 1, 40, 300, (60, 128)),
])
def test_calls_captured_together_equal_calls_one_by_one(H, dtype, B, Hq, Hkv, T, max_seq, lens):
    c = Calls(H, dtype, B, Hq, Hkv, max_seq, T)

    def new_inputs(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (c.q, c.qt, c.x):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        c.long.copy_(torch.randint(lens[0], lens[1] + 1, (B,), generator=g, device="cuda") if seed % 2 else i32([lens[1]] * B))
        c.short.copy_(torch.randint(T, max(T, lens[0] // 2) + 1, (B,), generator=g, device="cuda"))

    new_inputs(0)
    for s in c.steps():
        s()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for s in c.steps():
            s()
    for seed in range(1, 13):
        new_inputs(seed)
        before = [t.clone() for t in c.state()]
        for s in c.steps():
            s()
            torch.cuda.synchronize()
        want = [t.clone() for t in c.state()]
        for t, old in zip(c.state(), before):
            t.copy_(old)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(c.state(), want):
            assert torch.equal(got, w)
        for t, old in zip(c.state(), before):
            t.copy_(old)
        torch.cuda.synchronize()
        for s in c.steps():  # and enqueued one after another
            s()
        torch.cuda.synchronize()
        for got, w in zip(c.state(), want):
            assert torch.equal(got, w)
    for ws in (c.ws, c.pages_ws, c.status_ws):
        assert H.hata_read_device_status(ws) == 0

"""Calls of the MXFP4 and expert operators queued one behind another, without the host waiting between them.

Every kernel of these calls starts before the work ahead of it ends.  The chains below reuse all of their
buffers, so a kernel that read anything too early, or from an old copy of it, would give another result than
the same calls with the device synchronised after each; results are compared bit for bit.
"""
import numpy as np
import pytest

from oracle import mx
from test_gpu_experts import choices
from test_gpu_mxfp4 import on_gpu, q4q, rand  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


class Block:
    """Buffers of one mixture-of-experts block, and its calls."""

    def __init__(self, q4q, n, top, experts, k, rows, type_, seed):  # noqa: F811
        rng = np.random.default_rng(seed)
        self.q4q, self.n, self.top, self.experts, self.k, self.rows = q4q, n, top, experts, k, rows
        self.ids = [torch.from_numpy(choices(rng, n, top, experts)).cuda() for _ in range(3)]
        self.x = [on_gpu(rand(rng, n, k), type_)[0] for _ in range(3)]
        self.w32 = [torch.from_numpy(rng.standard_normal((experts, rows, k)).astype(np.float32) * 0.05).cuda() for _ in range(2)]
        self.weights = [torch.from_numpy(rng.random((n, top)).astype(np.float32)).cuda() for _ in range(3)]
        slots, dt = n * top, self.x[0].dtype
        size = q4q.q4q_mxfp4_size(k, rows)

        def new(*shape, dtype=dt):
            return torch.zeros(shape, dtype=dtype, device="cuda")
        self.first, self.slot, self.row = (new(m, dtype=torch.int32) for m in (experts + 1, slots, slots))
        self.packed = new(experts, size, dtype=torch.uint8)
        self.gathered, self.h, self.y = new(slots, k), new(slots, rows), new(n, rows)
        self.back, self.drows, self.dw = new(n, k), new(slots, rows), new(n, top, dtype=torch.float32)
        self.decoded = new(rows, k, dtype=torch.float32)
        self.ws = new(q4q.q4q_mul_mat_id_mxfp4_workspace_size(k, rows, n, slots, experts), dtype=torch.uint8)
        self.outputs = (self.first, self.slot, self.row, self.packed, self.gathered, self.h, self.y, self.back, self.drows, self.dw, self.decoded)

    def step(self, i, wait=lambda: None, stream=None):
        """Every operator once, on the inputs of turn i, into the same buffers as every other turn."""
        q, ids, x, w = self.q4q, self.ids[i % 3], self.x[i % 3], self.weights[i % 3]
        s = {"stream": stream}
        calls = (
            lambda: q.q4q_quantize_mxfp4(self.w32[i % 2], self.packed, **s),
            lambda: q.q4q_get_rows_mxfp4(self.packed[0], self.k, self.rows, dst=self.decoded, **s),
            lambda: q.q4q_moe_sort(ids, self.experts, self.first, self.slot, self.row, **s),
            lambda: q.q4q_moe_gather(x, self.first, self.row, self.top, self.gathered, **s),
            lambda: q.q4q_mul_mat_id_mxfp4(self.packed, self.k, self.rows, x, self.first, self.slot, self.top, dst=self.h, workspace=self.ws, **s),
            lambda: q.q4q_moe_combine(self.h, self.first, self.row, w, self.y, **s),
            lambda: q.q4q_moe_gather_back(self.gathered, self.first, self.row, self.top, self.back, **s),
            lambda: q.q4q_moe_combine_back(self.y, self.h, self.first, self.row, w, self.drows, self.dw, **s))
        for call in calls:
            call()
            wait()

    def waited(self):
        """The outputs of turns 0 to 5 with the device synchronised after every call."""
        out = []
        for i in range(6):
            self.step(i, torch.cuda.synchronize)
            out.append([t.clone() for t in self.outputs])
        torch.cuda.synchronize()
        return out


SIZES = [(1, 2, 8, 256, 160, "f32"), (37, 4, 6, 288, 96, "bf16"), (300, 2, 16, 512, 260, "f16")]


def same(got, ref, what):
    for g, r in zip(got, ref):
        assert torch.equal(g, r), what


@pytest.mark.parametrize("n,top,experts,k,rows,type_", SIZES)
def test_queued_calls_that_reuse_every_buffer(q4q, n, top, experts, k, rows, type_):  # noqa: F811
    b = Block(q4q, n, top, experts, k, rows, type_, [n, k])
    ref = b.waited()
    got = []
    for i in range(60):
        b.step(i)
        got.append([t.clone() for t in b.outputs] if i % 7 == 0 or i > 53 else None)
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        if g is not None:
            same(g, ref[i % 6], "turn %d" % i)
    assert q4q.q4q_device_status() == 0


@pytest.mark.parametrize("tokens,type_", [(1, "f32"), (20, "bf16"), (130, "f16")])
def test_chain_of_products_in_place(q4q, tokens, type_):  # noqa: F811
    """Each product reads the matrix that it replaces."""
    rng = np.random.default_rng(tokens)
    w = [torch.from_numpy(mx.pack((rng.standard_normal((256, 256)) / 16).astype(np.float32))[0]).cuda() for _ in range(3)]
    x = on_gpu(rand(rng, tokens, 256), type_)[0]
    ref, got = x.clone(), x.clone()
    ws = torch.empty(q4q.q4q_mul_mat_mxfp4_workspace_size(256, 256, tokens), dtype=torch.uint8, device="cuda")
    for i in range(40):
        q4q.q4q_mul_mat_mxfp4(w[i % 3], 256, 256, ref, dst=ref, workspace=ws)
        torch.cuda.synchronize()
    for i in range(40):
        q4q.q4q_mul_mat_mxfp4(w[i % 3], 256, 256, got, dst=got, workspace=ws)
    torch.cuda.synchronize()
    assert torch.isfinite(ref).all() and float(ref.abs().max()) > 0
    assert torch.equal(got, ref)


@pytest.mark.parametrize("n,top,experts,k,rows,type_", SIZES)
def test_calls_on_another_stream(q4q, n, top, experts, k, rows, type_):  # noqa: F811
    b = Block(q4q, n, top, experts, k, rows, type_, [n, k, 1])
    ref = b.waited()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for i in range(6):
        b.step(i, stream=side)
        with torch.cuda.stream(side):
            got.append([t.clone() for t in b.outputs])
    side.synchronize()
    for i in range(6):
        same(got[i], ref[i], "turn %d" % i)


def new_results(b, i, stream=None):
    """The same calls with results and workspaces of their own."""
    q, ids, x, w, s = b.q4q, b.ids[i % 3], b.x[i % 3], b.weights[i % 3], {"stream": stream}
    packed = q.q4q_quantize_mxfp4(b.w32[i % 2], **s)
    decoded = q.q4q_get_rows_mxfp4(packed[0], b.k, b.rows, **s)
    first, slot, row = q.q4q_moe_sort(ids, b.experts, **s)
    gathered = q.q4q_moe_gather(x, first, row, b.top, **s)
    h = q.q4q_mul_mat_id_mxfp4(packed, b.k, b.rows, x, first, slot, b.top, **s)
    y = q.q4q_moe_combine(h, first, row, w, **s)
    back = q.q4q_moe_gather_back(gathered, first, row, b.top, **s)
    drows, dw = q.q4q_moe_combine_back(y, h, first, row, w, **s)
    return first, slot, row, packed, gathered, h, y, back, drows, dw, decoded


@pytest.mark.parametrize("n,top,experts,k,rows,type_", SIZES)
def test_new_results_on_another_stream(q4q, n, top, experts, k, rows, type_):  # noqa: F811
    b = Block(q4q, n, top, experts, k, rows, type_, [n, k, 2])
    ref = b.waited()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [new_results(b, i, side) for i in range(6)]
    torch.cuda.current_stream().wait_stream(side)
    for i in range(6):
        same(got[i], ref[i], "turn %d" % i)


@pytest.mark.parametrize("n,top,experts,k,rows,type_", SIZES)
def test_calls_in_a_graph(q4q, n, top, experts, k, rows, type_):  # noqa: F811
    """Two turns in one graph, into the block's buffers and into the graph's own memory."""
    b = Block(q4q, n, top, experts, k, rows, type_, [n, k, 3])
    ref = b.waited()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.step(0)
        own = new_results(b, 1)
        b.step(5)
    for _ in range(3):
        for t in b.outputs + own:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        same(b.outputs, ref[5], "buffers")
        same(own, ref[1], "the graph's memory")
    assert q4q.q4q_device_status() == 0

"""A decode step of sequences that share a prompt, as a server runs it: 8-bit projections of quantised activations, the new
tokens' latents into the cache, attention behind the shared prefix, the output projection, a gate in 8 bits, selection with
groups and the routed experts.  Each operator is checked against its formula on what it was given in the run (tolerances:
each operator's own test), and the step as a captured graph, whose sequences grow from replay to replay, against the same
calls made one by one."""
import pytest
import torch

import oracle
import synth
from synth.device import upload_layer
from tests import mla_ref as ref
from tests.gpu_util import parity, q, say, status
from tests.test_gpu_select import reference as select_reference
from tests.test_gpu_shared import reference as shared_reference
from tests.test_gpu_w8 import BF, F32, TINY, U, codes_of, exact_sums

pytestmark = pytest.mark.gpu

RANK, NOPE, V, PAGE, SPEC = 256, 128, 128, 16, synth.TINY
HIDDEN = SPEC.hidden


@pytest.fixture(scope="module", autouse=True)
def device():
    assert torch.cuda.is_available(), "no GPU visible"


@pytest.fixture(params=["together", "apart"], autouse=True)
def path(request, device):
    """Both ways to read the prefix: at these sizes the choice between them is always the second."""
    q().coli_mla_debug_shared_path({"together": 1, "apart": 2}[request.param])
    yield request.param
    q().coli_mla_debug_shared_path(0)


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class Server:
    """Weights, cache and workspaces; `kept` holds what each operator of the last step got and gave."""

    def __init__(self, lens, prefix, heads, fp8, room=8):
        m, g = q(), torch.Generator(device="cuda").manual_seed(prefix + heads)
        self.n, self.prefix, self.heads, self.max_kv = len(lens), prefix, heads, max(lens) + room

        def randn(*shape):
            return torch.randn(shape, generator=g, device="cuda")

        def weight(rows, k):
            codes, scale = torch.empty(rows, k, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
            m.coli_w8_quantize(randn(rows, k) / k ** 0.5, codes, scale)
            return codes, scale
        self.w_q, self.w_kv_a = weight(heads * (NOPE + 64), HIDDEN), weight(RANK + 64, HIDDEN)
        self.w_o, self.w_gate = weight(HIDDEN, heads * V), weight(SPEC.n_experts, HIDDEN)
        self.w_k_t, self.w_v = (randn(heads, RANK, NOPE) / 8).to(BF), (randn(heads, V, RANK) / 16).to(BF)
        self.gain, self.bias = torch.ones(RANK, dtype=BF, device="cuda"), 0.05 * randn(SPEC.n_experts)
        self.inv_freq = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64, device="cuda") / 64)
        self.dims = m.make_mla_dims(heads, RANK, NOPE, V, PAGE, BF, m.COLI_KV_E4M3 if fp8 else m.COLI_KV_PLAIN)
        shared, own = -(-prefix // PAGE), -(-self.max_kv // PAGE)
        n_pages = shared + self.n * own
        row = m.coli_mla_row_bytes(self.dims)
        self.pages = (torch.zeros(n_pages, PAGE, row, dtype=torch.uint8, device="cuda") if fp8
                      else torch.zeros(n_pages, PAGE, row // 2, dtype=BF, device="cuda"))
        self.kv_scale = torch.zeros(n_pages * PAGE, device="cuda") if fp8 else None
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        self.prefix_table, self.table = order[:shared].contiguous(), order[shared:].view(self.n, own).contiguous()
        self.ws = torch.zeros(m.coli_mla_shared_workspace_bytes(self.dims, self.n, 1, prefix, self.max_kv), dtype=torch.uint8,
                              device="cuda")
        self.layer_host = synth.tiny_layer(seed=1, S=1)
        self.layer = upload_layer(self.layer_host, device="cuda")
        self.select = m.make_select_dims(SPEC.n_experts, SPEC.top_k, 4, 2, m.COLI_SCORE_SIGMOID, m.COLI_GROUP_TOP2, True, 2.5)
        self.moe_dims = m.make_dims(SPEC)
        self.moe_ws = torch.zeros(m.coli_moe_workspace_bytes(self.moe_dims, self.n), dtype=torch.uint8, device="cuda")
        # the prompt, then what each sequence holds before its next token
        self.fill(randn(prefix, RANK + 64), ref.slots_of(self.prefix_table[None], 0, prefix, PAGE), torch.arange(prefix, device="cuda"))
        for b, length in enumerate(lens):
            self.fill(randn(length, RANK + 64), ref.slots_of(self.table, b, length, PAGE),
                      prefix + torch.arange(length, device="cuda"))
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.x = torch.empty(self.n, HIDDEN, device="cuda")
        self.out = torch.empty(self.n, HIDDEN, device="cuda")
        self.kept = {}

    def fill(self, kv_a, slots, positions):
        if len(slots):
            q_pe = torch.zeros(len(slots), self.heads, 64, dtype=BF, device="cuda")
            q().coli_mla_append(self.dims, kv_a.to(BF), self.gain, positions.to(torch.int32), slots, self.inv_freq, q_pe, q_pe,
                                self.pages, self.kv_scale, self.ws)

    def linear(self, name, x, weight, dtype):
        n, k = x.shape
        codes, scale = torch.empty(n, k, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
        out = torch.empty(n, weight[0].shape[0], dtype=dtype, device="cuda")
        q().coli_w8_quantize(x, codes, scale)
        q().coli_w8_linear(codes, scale, *weight, None, out)
        self.kept[name] = x, codes, scale, weight, out
        return out

    def step(self):
        """The next token of every sequence, from self.x to self.out."""
        m, n, heads = q(), self.n, self.heads
        h = norm(self.x)
        queries, kv_a = self.linear("q", h, self.w_q, BF).view(n, heads, NOPE + 64), self.linear("kv_a", h, self.w_kv_a, BF)
        at = self.lens.long()
        slots = self.table.long().gather(1, (at // PAGE)[:, None])[:, 0] * PAGE + at % PAGE
        q_pe = torch.empty(n, heads, 64, dtype=BF, device="cuda")
        m.coli_mla_append(self.dims, kv_a, self.gain, self.lens + self.prefix, slots, self.inv_freq, queries[..., NOPE:], q_pe,
                          self.pages, self.kv_scale, self.ws)
        self.lens += 1
        q_lat, o_lat = (torch.empty(n, heads, RANK, dtype=BF, device="cuda") for _ in range(2))
        attended = torch.empty(n, heads, V, dtype=BF, device="cuda")
        m.coli_mla_project(queries[..., :NOPE], self.w_k_t, q_lat)
        m.coli_mla_decode_shared(self.dims, q_lat, q_pe, self.pages, self.kv_scale, self.prefix_table, self.prefix, self.table,
                                 self.lens, self.max_kv, o_lat, None, self.ws)
        m.coli_mla_project(o_lat, self.w_v, attended)
        x = self.x + self.linear("o", attended.view(n, heads * V), self.w_o, F32)
        h = norm(x)
        logits = self.linear("gate", h, self.w_gate, F32)
        idx = torch.empty(n, SPEC.top_k, dtype=torch.int32, device="cuda")
        w, out = torch.empty(n, SPEC.top_k, device="cuda"), torch.empty(n, HIDDEN, device="cuda")
        m.coli_moe_select(self.select, logits, self.bias, idx, w, self.moe_ws)
        m.coli_moe_forward(self.moe_dims, h, idx, w, self.layer["table"], self.layer["shared"], out, self.moe_ws)
        torch.add(x, out, out=self.out)
        self.kept.update(attend=(q_lat, q_pe, o_lat), select=(logits, idx, w), experts=(h, idx, w, out))

    def ok(self):
        assert status(self.ws) == 0 and status(self.moe_ws) == 0, q().coli_moe_last_error()

    def check(self):
        """The last step's operators against their formulas."""
        for name in ("q", "kv_a", "o", "gate"):
            x, codes, scale, (w, w_scale), out = self.kept[name]
            top = x.double().abs().amax(-1) / 127.0
            assert torch.equal(scale, top.float()) and torch.equal(codes, codes_of(x, scale)), name
            want = exact_sums(codes, w) * scale.double()[:, None] * w_scale.double()
            u = 0.0 if out.dtype == F32 else U[out.dtype]
            ref.close(out, want, (4.02 * ref.U32 + 1.01 * u) * want.abs() + 4 * 2.0 ** -149 + TINY[out.dtype], name)
        q_lat, q_pe, o_lat = self.kept["attend"]
        lat, key = ref.rows_of(self.pages, self.kv_scale, RANK, BF)
        lens = self.lens.tolist()
        want, _, mag, smag = shared_reference(q_lat, q_pe, lat, key, self.prefix_table, self.prefix, self.table, lens, 1, PAGE,
                                              self.dims.softmax_scale)
        ref.close(o_lat, want, ref.attend_tol(want, mag, smag, RANK + 64, self.prefix + max(lens), BF)[0], "attention")
        logits, idx, w = self.kept["select"]
        want_idx, want_w = select_reference(self.select, logits, self.bias)
        assert (idx.cpu().numpy() == want_idx).all()
        assert (abs(w.double().cpu().numpy() - want_w) <= 2.0 ** -24 * 1.001 * abs(want_w)).all()
        h, idx, w, out = (t.cpu().numpy() for t in self.kept["experts"])
        parity(out, oracle.forward(SPEC, h, idx, w, self.layer_host["blobs"], self.layer_host["shared"]))


CASES = [([0], 1, 8, False), ([3, 0, 17, 40, 31], 100, 8, False), ([3, 0, 17, 40, 31], 100, 8, True),
         ([5, 64, 0], 333, 128, False), ([60, 1, 1, 1, 15, 16, 17], 500, 128, True)]


@pytest.mark.parametrize("lens,prefix,heads,fp8", CASES)
def test_step(lens, prefix, heads, fp8):
    say("serving step", lens, prefix, heads, fp8)
    server, g = Server(lens, prefix, heads, fp8), torch.Generator(device="cuda").manual_seed(7)
    for _ in range(2):
        server.x.copy_(torch.randn(server.n, HIDDEN, generator=g, device="cuda"))
        server.step()
        server.ok()
        server.check()


@pytest.mark.parametrize("lens,prefix,heads,fp8", CASES)
def test_step_captured(lens, prefix, heads, fp8):
    say("serving step captured", lens, prefix, heads, fp8)
    eager, graphed = Server(lens, prefix, heads, fp8), Server(lens, prefix, heads, fp8)
    g = torch.Generator(device="cuda").manual_seed(8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    first = torch.randn(eager.n, HIDDEN, generator=g, device="cuda")
    with torch.cuda.stream(side):   # on a stream of its own once, as before any capture
        graphed.x.copy_(first)
        graphed.step()
    side.synchronize()
    eager.x.copy_(first)
    eager.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.step()
    for _ in range(4):
        x = torch.randn(eager.n, HIDDEN, generator=g, device="cuda")
        eager.x.copy_(x)
        eager.step()
        graphed.x.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager.out, graphed.out) and torch.equal(eager.lens, graphed.lens)
        assert torch.equal(eager.pages, graphed.pages)
    for server in (eager, graphed):
        server.ok()
    eager.check()


def test_two_steps_at_once():
    """Two batches on two streams, each with its own workspaces, beside one another."""
    say("two serving steps")
    servers = [Server([3, 0, 17, 40, 31], 100, 8, False), Server([5, 64, 0], 333, 128, False)]
    alone = [Server([3, 0, 17, 40, 31], 100, 8, False), Server([5, 64, 0], 333, 128, False)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    g = torch.Generator(device="cuda").manual_seed(9)
    for _ in range(3):
        for server, other in zip(servers, alone):
            server.x.copy_(torch.randn(server.n, HIDDEN, generator=g, device="cuda"))
            other.x.copy_(server.x)
            other.step()
        torch.cuda.synchronize()
        for server, stream in zip(servers, streams):
            with torch.cuda.stream(stream):
                server.step()
        torch.cuda.synchronize()
        for server, other in zip(servers, alone):
            server.ok()
            assert torch.equal(server.out, other.out)

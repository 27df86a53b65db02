"""The serving step's operators between other work on their streams: captured behind copies, sets
and a join of two streams, and verification where every sequence is left out, with its workspace
and its logits used again at once."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_deltanet_linear_13_gb300 as m
    from gated_deltanet_linear_13_gb300 import build_lib
    build_lib.build()
    m.load_library()
    return m


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


class Step:
    """A plan, the norm and rotation into the planned slots, a verification, a release."""

    def __init__(self, gdn, seed):
        i32 = dict(device="cuda", dtype=torch.int32)
        g = _gen(seed)
        self.gdn, b, t, d, v = gdn, 5, 2, 128, 3001
        self.pool = dict(table=torch.zeros(b, 8, **i32), held=torch.zeros(b, **i32),
                         free_pages=torch.randperm(40, generator=g, device="cuda").to(torch.int32),
                         free_count=torch.full((1,), 40, **i32), page_size=16)
        self.length = torch.tensor([0, 7, 15, 16, 90], **i32)
        self.new = torch.tensor([3, 0, 1, 3, 2], **i32)
        self.slots, self.positions = torch.zeros(12, **i32), torch.zeros(12, **i32)
        self.q = torch.randn(12, 6, d, generator=g, device="cuda").bfloat16()
        self.k = torch.randn(12, 2, d, generator=g, device="cuda").bfloat16()
        self.q_out = torch.zeros_like(self.q)
        self.k_cache = torch.zeros(40, 2, 16, d, device="cuda", dtype=torch.bfloat16)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.steps, self.amplitude = gdn.gdn_rope_phase_steps(64)
        self.logits = torch.randn(b, t + 1, v, generator=g, device="cuda")
        self.ids = self.logits[:, :t].argmax(-1).to(torch.int32)
        self.u = torch.rand(b, t, generator=g, device="cuda")
        self.clocks = torch.empty(b, v, device="cuda").exponential_(generator=g)
        self.tokens, self.accepted = torch.zeros(b, t + 1, **i32), torch.zeros(b, **i32)
        self.workspace = torch.full((gdn.gdn_verify_tokens_workspace_size(
            b, t, v, torch.float32, False),), 255, device="cuda", dtype=torch.uint8)

    def plan(self):
        self.gdn.gdn_page_plan(self.length, self.new, self.slots, self.positions, **self.pool)

    def rotate(self):
        self.gdn.gdn_qk_norm_rope(self.q, self.k, self.positions, self.steps, self.q_out, v=self.k,
                                  k_cache=self.k_cache, v_cache=self.v_cache, slots=self.slots)

    def verify(self):
        self.gdn.gdn_verify_tokens(self.logits, self.tokens, self.accepted, clocks=self.clocks,
                                   draft_ids=self.ids, accept_u=self.u, workspace=self.workspace)

    def release(self):
        self.gdn.gdn_page_release(self.length, **self.pool)

    def state(self):
        return [x.clone() for x in (self.pool["table"], self.pool["held"], self.pool["free_pages"],
                                    self.pool["free_count"], self.slots, self.positions, self.q_out,
                                    self.k_cache, self.v_cache, self.tokens, self.accepted)]


def _all(step, between):
    for call in (step.plan, step.rotate, step.verify, step.release):
        between()
        call()
    between()


def test_captured_between_other_nodes(gdn):
    """Copies, sets and torch's kernels before each call, and a second stream that forks before it
    and joins behind: the replays give what the plain calls give."""
    want = Step(gdn, 3)
    _all(want, lambda: None)
    torch.cuda.synchronize()
    step = Step(gdn, 3)
    source = torch.randn(1 << 20, device="cuda")
    target, host = torch.zeros_like(source), torch.zeros(1 << 10).pin_memory()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    kinds = (lambda: target.copy_(source), lambda: target.zero_(), lambda: target.add_(1.0),
             lambda: host.copy_(source[:1 << 10], non_blocking=True))

    def fork(work):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            work()
        kinds[2]()
        torch.cuda.current_stream().wait_stream(side)

    graphs = []
    for work in (*kinds, *(lambda k=k: fork(k) for k in kinds)):
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=main):
            _all(step, work)
        graphs.append(graph)
    first = step.state()
    for graph in graphs:
        for x, y in zip((step.pool["table"], step.pool["held"], step.pool["free_pages"],
                         step.pool["free_count"], step.slots, step.positions, step.q_out,
                         step.k_cache, step.v_cache, step.tokens, step.accepted), first):
            x.copy_(y)
        torch.cuda.synchronize()
        with torch.cuda.stream(main):
            graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(step.state(), want.state()):
            assert torch.equal(x, y)
    assert gdn.gdn_get_device_error() == 0


@pytest.mark.parametrize("drafts", [0, 2])
def test_nothing_taken_then_all(gdn, drafts):
    """Calls that leave every sequence out write nothing but the workspace, and are over before
    what comes behind them: a call with the same workspace, and new logits."""
    b, v = 40, 60000
    g = _gen(drafts)
    a, z = (torch.randn(b, drafts + 1, v, generator=g, device="cuda").bfloat16() for _ in range(2))
    x = a.clone()
    c = dict(clocks=torch.empty(b, v, device="cuda").exponential_(generator=g))
    if drafts:
        c.update(draft_ids=a[:, :drafts].float().argmax(-1).to(torch.int32),
                 accept_u=torch.rand(b, drafts, generator=g, device="cuda"))
    ws = torch.full((gdn.gdn_verify_tokens_workspace_size(b, drafts, v, torch.bfloat16, False),),
                    255, device="cuda", dtype=torch.uint8)
    none, every = torch.zeros(b, device="cuda"), torch.ones(b, device="cuda")
    i32 = dict(device="cuda", dtype=torch.int32)

    def run(logits, scale, **kw):
        out = torch.full((b, drafts + 1), -9, **i32), torch.full((b,), -9, **i32)
        gdn.gdn_verify_tokens(logits, *out, scale=scale, **c, **kw)
        return out

    want_a, want_z = run(a, every), run(z, every)
    torch.cuda.synchronize()
    for _ in range(20):
        outs = [run(x, none, workspace=ws), run(x, every, workspace=ws),
                run(x, none, workspace=ws)]
        x.copy_(z)
        outs.append(run(x, every, workspace=ws))
        x.copy_(a)
        torch.cuda.synchronize()
        for out in (outs[0], outs[2]):
            assert all(int((o != -9).sum()) == 0 for o in out)
        assert all(torch.equal(o, w) for o, w in zip(outs[1], want_a))
        assert all(torch.equal(o, w) for o, w in zip(outs[3], want_z))
    assert gdn.gdn_get_device_error() == 0

"""Prompt, replayed steps, verification and flushes together, as a decode loop
runs them: nothing read back on the host between them, and the same captured
in HIP graphs, on streams of their own and interleaved."""
import pytest
import torch

from tests import delta_refs as R

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import speculative_replay_state_amd as ssu
    from tests import gpu_harness as gh
    import synth
    from synth import device as sd

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


class Loop:
    """Requests of one layer: a prompt each, then steps of T tokens whose
    acceptance comes from given probabilities."""

    def __init__(self, seed, batch=5, T=4, steps=6, hk=2, hv=4, dk=64, dv=64, L=16, state="f32", vocab=50):
        g = gen(seed)
        self.batch, self.T, self.steps, self.hk, self.hv, self.dk, self.dv, self.L, self.vocab = batch, T, steps, hk, hv, dk, dv, L, vocab
        self.state = state
        self.lens = torch.randint(0, 70, (batch,), generator=g).tolist()
        cu = [0]
        for n in self.lens:
            cu.append(cu[-1] + n)
        self.cu = cu
        self.prompt = R.inputs(g, cu[-1], hk, hv, dk, dv)
        self.new = []
        for _ in range(steps):
            x = R.inputs(g, batch * T, hk, hv, dk, dv)
            x["A"], x["dt_bias"] = self.prompt["A"], self.prompt["dt_bias"]
            self.new.append(x)
        self.tokens = torch.randint(0, vocab, (steps, batch * T), generator=g, dtype=torch.int32)
        self.probs = torch.softmax(torch.randn(steps, batch * T, vocab, generator=g), -1)
        self.u = 0.03 * torch.rand(steps, batch * T, generator=g)
        self.uf = torch.rand(steps, batch, generator=g)
        self.ids = (1 + torch.randperm(batch + 2, generator=g)[:batch]).to(torch.int32)

    def build(self):
        """Device tensors and the calls of one pass over the loop."""
        z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt, device=DEV)  # noqa: E731
        i32 = torch.int32
        slots, b, T = self.batch + 3, self.batch, self.T
        size = R.TYPES[self.state].itemsize
        self.d = dict(state=z(slots, self.hv * self.dv * self.dk * size), k_cache=z(slots, self.hk * self.L * self.dk * 2),
                      v_cache=z(slots, self.hv * self.L * self.dv * 2), gate_cache=z(slots, self.hv * self.L * 8),
                      ring_start=z(slots, dt=i32), status=z(1, dt=i32))
        d = self.d
        self.dc = ssu.DeltaCache(slots, self.hk, self.hv, self.L, self.state, d["state"], d["k_cache"], d["v_cache"], d["gate_cache"],
                                 d["ring_start"], d["status"], dim_k=self.dk, dim_v=self.dv)
        up = lambda x: {k: v.to(DEV) for k, v in x.items()}  # noqa: E731
        p = up(self.prompt)
        rows = self.cu[-1]
        self.prompt_out = z(rows, self.hv, self.dv, dt=torch.float32)
        self.final = z(b, self.hv, self.dv, self.dk, dt=torch.float32)
        ws = z(max(16, ssu.delta_prefill_workspace_size(rows, b, self.hv)))
        self.slot_idx = self.ids.to(DEV)
        pre = ssu.make_delta_prefill(torch.tensor(self.cu, dtype=i32, device=DEV), p["q"], p["k"], p["v"], p["dt"], p["beta"], p["A"],
                                     p["dt_bias"], self.prompt_out, final_states=self.final, workspace=ws)
        self.left, self.live, self.fold = z(b, dt=i32), z(b, dt=i32), z(b, dt=i32)
        self.outs, self.acc, self.toks, self.folds, self.calls = [], [], [], [], [pre]
        vws = z(max(16, ssu.verify_workspace_size(b, self.vocab)))
        for s in range(self.steps):
            x = up(self.new[s])
            out, acc, tok = z(b * T, self.hv, self.dv, dt=torch.float32), z(b, dt=i32), z(b, T, dt=i32)
            step = ssu.make_delta_step(self.dc, T, self.slot_idx, self.left, None, x["q"], x["k"], x["v"], x["dt"], x["beta"], x["A"],
                                       x["dt_bias"], out)
            ver = ssu.make_verify(self.tokens[s].to(DEV), self.probs[s].to(DEV), None, self.u[s].to(DEV), self.uf[s].to(DEV), tok, acc,
                                  vws, live=self.left, ring_len=self.L, next_live=self.live, next_fold=self.fold,
                                  next_left=self.left)
            self.calls.append((step, ver))
            self.outs.append(out), self.acc.append(acc), self.toks.append(tok), self.folds.append(z(b, dt=i32))

    def reset(self):
        self.left.zero_()
        self.d["status"].zero_()
        for o in self.outs:
            o.zero_()

    def run(self, stream=None):
        ssu.delta_prefill(self.calls[0], stream)
        ssu.delta_init_state(self.dc, self.final, self.slot_idx, stream)
        for s, (step, ver) in enumerate(self.calls[1:]):
            ssu.delta_replay_step(self.dc, step, stream)
            ssu.verify(ver, stream)
            ssu.delta_flush(self.dc, self.slot_idx, self.fold, stream)
            self.folds[s].copy_(self.fold)

    def results(self):
        return [self.prompt_out, self.final, *self.outs, *self.acc, *self.toks, *self.folds, *[self.d[n] for n in sorted(self.d)], self.left]

    def check(self):
        """Against the rule over each request's kept tokens."""
        assert int(self.d["status"]) == 0
        gp = R.gates(self.prompt["dt"], self.prompt["beta"], self.prompt["A"], self.prompt["dt_bias"])
        folded = 0
        for j in range(self.batch):
            at = slice(self.cu[j], self.cu[j + 1])
            S, _ = R.run(torch.zeros(self.hv, self.dv, self.dk), None, *(self.prompt[n][at] for n in ("k", "v")), gp[0][at], gp[1][at], 1.0)
            n = self.lens[j]
            mass = self.prompt["v"][at].double().norm()
            for s in range(self.steps):
                x = self.new[s]
                g, b = R.gates(x["dt"], x["beta"], x["A"], x["dt_bias"])
                rows = slice(j * self.T, (j + 1) * self.T)
                _, o = R.run(S, x["q"][rows], x["k"][rows], x["v"][rows], g[rows], b[rows], self.dk ** -0.5)
                mass = mass + x["v"][rows].double().norm()
                R.check(self.outs[s].cpu()[rows].transpose(0, 1), o.transpose(0, 1), self.dk ** -0.5 * float(mass),
                        R.tol(self.dk, 32, n // 32 + 2 + s, "f32"), "request %d step %d" % (j, s))
                kept = int(self.acc[s][j])
                keep = slice(j * self.T, j * self.T + kept)
                S, _ = R.run(S, None, x["k"][keep], x["v"][keep], g[keep], b[keep], 1.0)
                folded += int(self.folds[s][j])
        assert folded > 0
        assert len({int(a) for t in self.acc for a in t}) > 1


def test_a_decode_loop_of_prompt_steps_verification_and_flushes():
    loop = Loop(1)
    loop.build()
    loop.reset()
    loop.run()
    torch.cuda.synchronize()
    loop.check()


def test_the_loop_in_a_graph_replayed_between_eager_runs():
    loop, other = Loop(2, L=32, steps=9, state="bf16"), Loop(2, L=32, steps=9, state="bf16")
    loop.build(), other.build()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    loop.reset()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        loop.run()
    for _ in range(3):
        other.reset()
        other.run()
        torch.cuda.synchronize()
        want = [t.clone() for t in other.results()]
        loop.reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(loop.results(), want))
        for t in loop.results():
            t.zero_()


def test_loops_interleaved_on_streams_of_their_own():
    loops = [Loop(3 + i, batch=3 + 4 * i, state=("f32", "f16", "bf16")[i], dk=(64, 128, 64)[i]) for i in range(3)]
    want = []
    for l in loops:
        l.build()
        l.reset()
        l.run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in l.results()])
        l.reset()
    streams = [torch.cuda.Stream() for _ in loops]
    torch.cuda.synchronize()
    for l, s in zip(loops, streams):
        with torch.cuda.stream(s):
            ssu.delta_prefill(l.calls[0])
            ssu.delta_init_state(l.dc, l.final, l.slot_idx)
    for i in range(max(l.steps for l in loops)):
        for l, s in zip(loops, streams):
            step, ver = l.calls[1 + i]
            ssu.delta_replay_step(l.dc, step, s)  # the stream as an argument
            ssu.verify(ver, s)
            ssu.delta_flush(l.dc, l.slot_idx, l.fold, s)
            with torch.cuda.stream(s):
                l.folds[i].copy_(l.fold)
    torch.cuda.synchronize()
    for l, w in zip(loops, want):
        assert all(torch.equal(a, b) for a, b in zip(l.results(), w))


def test_two_graphs_replayed_at_once():
    """Two captured loops, caches and scratch of their own, replayed on two streams without a wait between them."""
    loops = [Loop(11, batch=6, L=16, state="bf16", dk=128), Loop(12, batch=9, L=32, steps=5, state="f32")]
    graphs, want = [], []
    for l in loops:
        l.build()
        l.reset()
        l.run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in l.results()])
        l.reset()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=torch.cuda.Stream()):
            l.run()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for l in loops:
            for t in l.results():
                t.zero_()
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for l, w in zip(loops, want):
            assert all(torch.equal(a, b) for a, b in zip(l.results(), w))


def test_verification_drives_the_selective_state_update():
    """next_live and next_fold are the prev_num_accepted and num_fold of the next fused ssu step: a loop of them
    equals steps and flushes whose counts the host keeps."""
    spec = synth.CacheSpec(num_slots=9, nheads=16, ngroups=2, state_dtype="f32", ring_len=16)
    cache = synth.make_cache(spec, 21)
    b, T, vocab = 6, 4, 64
    g = gen(22)
    steps = [synth.make_step(spec, b, T, 30 + i, 0) for i in range(16)]
    ids = steps[0].slot_idx
    t1, t2 = sd.upload_cache(cache, DEV), sd.upload_cache(cache, DEV)
    c1, c2 = gh.device_cache(spec, t1), gh.device_cache(spec, t2)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    live, fold = i32([0] * b), i32([0] * b)
    ws = torch.empty(max(16, ssu.verify_workspace_size(b, vocab)), dtype=torch.uint8, device=DEV)
    host_live = [0] * b
    slots = torch.from_numpy(ids).to(DEV)
    folded = 0
    for i, s in enumerate(steps):
        st = sd.upload_step(s, DEV)
        o1, o2 = gh.out_tensor(s, spec, "f32"), gh.out_tensor(s, spec, "f32")
        desc = ssu.make_step_desc(b, T, slots, live, None, st["x"], st["B"], st["C"], st["dt"], st["A"], st["D"], st["dt_bias"], o1,
                                  "f32", num_fold=fold)
        ssu.replay_step(c1, desc)
        tokens = torch.randint(0, vocab, (b * T,), generator=g, dtype=torch.int32)
        probs = torch.softmax(torch.randn(b * T, vocab, generator=g), -1)
        u = 0.02 * torch.rand(b * T, generator=g)
        out, acc = torch.empty(b, T, dtype=torch.int32, device=DEV), torch.empty(b, dtype=torch.int32, device=DEV)
        ssu.verify(ssu.make_verify(tokens.to(DEV), probs.to(DEV), None, u.to(DEV), torch.rand(b, generator=g).to(DEV), out, acc, ws,
                                   live=live, fold=fold, ring_len=16, reserve=2 * T, next_live=live, next_fold=fold))
        # the host's own bookkeeping: flush first, then a plain step
        k = [n if n + 2 * T > 16 else 0 for n in host_live]
        folded += sum(k)
        ssu.flush(c2, slots, i32(k), st["A"])
        host_live = [n - f for n, f in zip(host_live, k)]
        ssu.replay_step(c2, ssu.make_step_desc(b, T, slots, i32(host_live), None, st["x"], st["B"], st["C"], st["dt"], st["A"], st["D"],
                                               st["dt_bias"], o2, "f32"))
        host_live = [n + a for n, a in zip(host_live, acc.tolist())]
        assert live.tolist() == host_live
        assert torch.equal(o1, o2), "step %d" % i
    assert folded > 0
    assert torch.equal(t1["state"], t2["state"]) and torch.equal(t1["ring_start"], t2["ring_start"])

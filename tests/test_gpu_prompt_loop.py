"""A decode loop as it is used, nothing read back on the host inside it: prompts
(prefill, init_state, their tokens counted), then steps, logits, verification,
counts and flushes, and the states read back at the end.  Eager, captured in
HIP graphs, on streams of its own."""
import numpy as np
import pytest
import torch

from tests import prompt_refs as R

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import speculative_replay_state_amd as ssu
    from tests import gpu_harness as gh
    from tests.test_gpu_logits import check_probs

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Loop:
    def __init__(self, seed, batch=5, T=4, steps=6, H=4, G=2, L=16, vocab=300, longest=150):
        g = torch.Generator()
        g.manual_seed(seed)
        self.batch, self.T, self.steps, self.H, self.G, self.L, self.vocab = batch, T, steps, H, G, L, vocab
        self.lens = (1 + torch.randint(0, longest, (batch,), generator=g)).tolist()
        self.cu = [sum(self.lens[:i]) for i in range(batch + 1)]
        self.prompt = R.inputs(g, self.cu[-1], H, G)
        self.prompt_tokens = torch.randint(0, vocab, (self.cu[-1],), generator=g, dtype=torch.int32)
        self.new = []
        for _ in range(steps):
            x = R.inputs(g, batch * T, H, G)
            x["A"], x["D"], x["dt_bias"] = (self.prompt[n] for n in ("A", "D", "dt_bias"))
            self.new.append(x)
        self.logits = 2.0 * torch.randn(steps, batch * T, vocab, generator=g)
        self.tokens = torch.randint(0, vocab, (steps, batch * T), generator=g, dtype=torch.int32)
        self.u = 0.9 / vocab * torch.rand(steps, batch * T, generator=g)   # (a part of the drafts is accepted)
        self.uf = torch.rand(steps, batch, generator=g)
        self.ids = (1 + torch.randperm(batch + 2, generator=g)[:batch]).to(torch.int32)
        self.rep, self.freq, self.pres = 1 + 0.3 * torch.rand(batch, generator=g), 0.2 * torch.rand(batch, generator=g), torch.rand(batch, generator=g)
        self.temperature = 0.7 + torch.rand(batch, generator=g)

    def build(self):
        z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt, device=DEV)  # noqa: E731
        f32, i32, b, T, H, G, L = torch.float32, torch.int32, self.batch, self.T, self.H, self.G, self.L
        slots, rows = b + 3, self.cu[-1]
        self.d = dict(state=z(slots, H * 64 * 128 * 4), x_cache=z(slots, H * L * 64 * 2), B_cache=z(slots, G * L * 128 * 2),
                      dt_cache=z(slots, H * L * 4), ring_start=z(slots, dt=i32), status=z(1, dt=i32))
        d = self.d
        self.cache = ssu.DeviceCache(slots, H, G, L, "f32", d["state"], None, d["x_cache"], d["B_cache"], d["dt_cache"], d["ring_start"],
                                     d["status"])
        self.counts, self.seen = z(slots, self.vocab, dt=i32), z(slots, (self.vocab + 31) // 32, dt=i32)
        history = ssu.TokenHistory(slots, self.vocab, self.counts, self.seen, d["status"])
        up = lambda x: {k: v.to(DEV) for k, v in x.items()}  # noqa: E731
        p = up(self.prompt)
        self.A = p["A"]
        self.prompt_out, self.final, self.back = z(rows, H, 64, dt=f32), z(b, H, 64, 128, dt=f32), z(b, H, 64, 128, dt=f32)
        cu, self.slot_idx = torch.tensor(self.cu, dtype=i32, device=DEV), self.ids.to(DEV)
        ws = z(max(16, ssu.prefill_workspace_size(rows, b, H)))
        self.pre = ssu.make_prefill(cu, p["x"], p["B"], p["C"], p["dt"], p["A"], p["D"], p["dt_bias"], self.prompt_out,
                                    final_states=self.final, workspace=ws, status=d["status"])
        self.first = ssu.make_count(history, self.slot_idx, self.prompt_tokens.to(DEV), cu_seqlens=cu, prompt=True, reset=True)
        self.left, self.live, self.fold = z(b, dt=i32), z(b, dt=i32), z(b, dt=i32)
        vws, lws = z(max(16, ssu.verify_workspace_size(b, self.vocab))), z(max(16, ssu.logits_workspace_size(b, T, self.vocab)))
        par = [t.to(DEV) for t in (self.temperature, self.rep, self.freq, self.pres)]
        self.calls, self.outs, self.probs, self.acc, self.toks, self.folds = [], [], [], [], [], []
        for s in range(self.steps):
            x = up(self.new[s])
            out, probs, acc, tok = z(b * T, H, 64, dt=f32), z(b * T, self.vocab, dt=f32), z(b, dt=i32), z(b, T, dt=i32)
            fed = self.tokens[s].to(DEV)
            step = ssu.make_step_desc(b, T, self.slot_idx, self.left, None, x["x"].contiguous(), x["B"].contiguous(), x["C"].contiguous(),
                                      x["dt"], x["A"], x["D"], x["dt_bias"], out, "f32")
            soft = ssu.make_logits(self.logits[s].to(DEV), probs, b, T, history=history, slot_idx=self.slot_idx, tokens=fed,
                                   temperature=par[0], repetition=par[1], frequency=par[2], presence=par[3], workspace=lws,
                                   status=d["status"])
            ver = ssu.make_verify(fed, probs, None, self.u[s].to(DEV), self.uf[s].to(DEV), tok, acc, vws, live=self.left, ring_len=L,
                                  next_live=self.live, next_fold=self.fold, next_left=self.left)
            self.calls.append((step, soft, ver, ssu.make_count(history, self.slot_idx, tok, num_tokens=acc)))
            for a, v in ((self.outs, out), (self.probs, probs), (self.acc, acc), (self.toks, tok), (self.folds, z(b, dt=i32))):
                a.append(v)

    def reset(self):
        self.left.zero_()
        self.d["status"].zero_()

    def begin(self, stream=None):
        ssu.prefill(self.pre, stream)
        ssu.init_state(self.cache, self.final, self.slot_idx, stream=stream)
        ssu.count(self.first, stream)

    def step(self, s, stream=None):
        step, soft, ver, count = self.calls[s]
        ssu.replay_step(self.cache, step, stream)
        ssu.logits(soft, stream)
        ssu.verify(ver, stream)
        ssu.count(count, stream)
        ssu.flush(self.cache, self.slot_idx, self.fold, self.A, stream)

    def end(self, stream=None):
        ssu.flush(self.cache, self.slot_idx, self.left, self.A, stream)
        ssu.read_state(self.cache, self.back, self.slot_idx, stream=stream)

    def run(self, stream=None):
        self.begin(stream)
        for s in range(self.steps):
            self.step(s, stream)
            self.folds[s].copy_(self.fold)
        self.end(stream)

    def results(self):
        return [self.prompt_out, self.final, self.back, *self.outs, *self.probs, *self.acc, *self.toks, *self.folds,
                *[self.d[n] for n in sorted(self.d)], self.left, self.seen, self.counts]

    def check(self):
        """Against the rules over each request's kept tokens."""
        assert int(self.d["status"]) == 0
        T, folded, longest = self.T, 0, 0
        pd, pg = R.gates(self.prompt["dt"], self.prompt["A"], self.prompt["dt_bias"])
        for j in range(self.batch):
            at = slice(self.cu[j], self.cu[j + 1])
            S0 = torch.zeros(self.H, 64, 128)
            seq = [self.prompt[n][at] for n in ("x", "B", "C")]
            S, _ = R.run(S0, *seq, pd[at], pg[at], self.prompt["D"])
            Sa, _ = R.run(S0, *(t.abs() for t in seq), pd[at], pg[at], self.prompt["D"].abs())
            n = self.lens[j]
            held = {int(i): 1 for i in self.prompt_tokens[at]}   # token -> 2 n + p
            for s in range(self.steps):
                x, rows = self.new[s], slice(j * T, (j + 1) * T)
                d, g = R.gates(x["dt"], x["A"], x["dt_bias"])
                seq = [x[k][rows] for k in ("x", "B", "C")]
                _, y = R.run(S, *seq, d[rows], g[rows], x["D"])
                _, ya = R.run(Sa, *(t.abs() for t in seq), d[rows], g[rows], x["D"].abs())
                got = self.outs[s].cpu()[rows].double()
                # a step's own bound, and what the state it began with may be off by
                allowed = gh.tol_for("f32", "f32") * (1 + y.abs()) + R.tol_state(n + T * s) * ya
                assert bool(((got - y).abs() <= allowed).all()), "request %d step %d" % (j, s)
                # the probabilities
                xs = self.logits[s][rows].numpy().copy()
                rep, freq, pres = (np.float32(v[j]) for v in (self.rep, self.freq, self.pres))
                for t in range(T):
                    times = {i: w >> 1 for i, w in held.items()}
                    for i in self.tokens[s][j * T + 1:j * T + t + 1].tolist():
                        times[i] = times.get(i, 0) + 1
                    for i, k in times.items():
                        v = xs[t, i] / rep if xs[t, i] > 0 else xs[t, i] * rep
                        xs[t, i] = v - (freq * np.float32(k) + (pres if k > 0 else np.float32(0)))
                check_probs(self.probs[s][rows].cpu(), xs, [float(self.temperature[j])] * T, "f32")
                # what was kept
                kept = int(self.acc[s][j])
                longest = max(longest, kept)
                emitted = self.toks[s][j, :kept].tolist()
                assert emitted[:-1] == self.tokens[s][j * T + 1:j * T + kept].tolist()
                for i in emitted:
                    held[i] = held.get(i, 0) + 2
                keep = slice(j * T, j * T + kept)
                seq = [x[k][keep] for k in ("x", "B", "C")]
                S, _ = R.run(S, *seq, d[keep], g[keep], x["D"])
                Sa, _ = R.run(Sa, *(t.abs() for t in seq), d[keep], g[keep], x["D"].abs())
                folded += int(self.folds[s][j])
            slot = int(self.ids[j])
            bits = np.unpackbits(self.seen[slot].cpu().numpy().view(np.uint8), bitorder="little")
            assert set(np.flatnonzero(bits).tolist()) == set(held)
            counts = self.counts[slot].cpu()
            assert all(int(counts[i]) == w for i, w in held.items())
            R.check(self.back[j], S, Sa, (2.0 ** -24, R.tol_state(n + T * self.steps) + 64 * 2.0 ** -24), "state of request %d" % j)
        assert folded > 0 and longest > 1


def test_a_decode_loop():
    loop = Loop(1)
    loop.build()
    loop.reset()
    loop.run()
    torch.cuda.synchronize()
    loop.check()


def test_prompts_in_segments_and_long_rows():
    loop = Loop(2, batch=3, T=3, steps=7, H=2, G=1, vocab=20011, longest=1500)
    loop.build()
    loop.reset()
    loop.run()
    torch.cuda.synchronize()
    loop.check()


def test_the_loop_in_a_graph_replayed_between_eager_runs():
    loop, other = (Loop(3, batch=6, steps=5, longest=1200, vocab=17001) for _ in range(2))
    loop.build(), other.build()
    graph = torch.cuda.CUDAGraph()
    loop.reset()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
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


def test_two_graphs_replayed_at_once():
    """Two captured loops, caches and scratch of their own, replayed on two streams without a wait between them."""
    loops = [Loop(4, batch=7, longest=1300), Loop(5, batch=4, L=32, steps=4, vocab=33000)]
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


def test_loops_interleaved_on_streams_of_their_own():
    loops = [Loop(6 + i, batch=3 + 2 * i, longest=(100, 1000, 300)[i]) for i in range(3)]
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
        l.begin(s)   # the stream as an argument
    for i in range(max(l.steps for l in loops)):
        for l, s in zip(loops, streams):
            with torch.cuda.stream(s):   # the current one
                l.step(i)
                l.folds[i].copy_(l.fold)
    for l, s in zip(loops, streams):
        l.end(s)
    torch.cuda.synchronize()
    for l, w in zip(loops, want):
        assert all(torch.equal(a, b) for a, b in zip(l.results(), w))

"""Steps with a tree of drafts as a server runs them: a small model generates
with trees of drafts, and what it emits is what it emits token by token
without drafts; captured and replayed; several at once on streams and in
threads."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
B, N, V, D, HQ, HKV, LAYERS, L = 4, 12, 61, 16, 6, 2, 3, 96
HIDDEN = HQ * D


def sv():
    import speculative_sampling_verification_vocab_amd as m
    return m


class Model:
    """Embeddings with positions, attention layers with residuals, and a head."""

    def __init__(self, dtype=torch.float64):
        g = torch.Generator().manual_seed(1)

        def w(*shape):
            return torch.randn(shape, generator=g, dtype=torch.float64) * shape[0] ** -0.5
        self.embed, self.place, self.out = w(V, HIDDEN) * V ** 0.5, w(L + N, HIDDEN) * L ** 0.5, w(HIDDEN, V) * 2
        self.layers = [[w(HIDDEN, HQ * D) * 3, w(HIDDEN, HKV * D), w(HIDDEN, HKV * D), w(HIDDEN, HIDDEN) * 2]
                       for _ in range(LAYERS)]

    def to(self, dtype, device):
        m = object.__new__(Model)
        m.embed, m.place, m.out = (x.to(device, dtype) for x in (self.embed, self.place, self.out))
        m.layers = [[x.to(device, dtype) for x in y] for y in self.layers]
        return m

    def head(self, x):
        return x @ self.out

    def plain(self, tokens):
        """Logits after the last of `tokens`, in 64 bits."""
        n = len(tokens)
        x = self.embed[tokens] + self.place[:n]
        mask = torch.ones(n, n, dtype=torch.bool).tril()
        for wq, wk, wv, wo in self.layers:
            q = (x @ wq).view(n, HKV, HQ // HKV, D)
            k, v = (x @ wk).view(n, HKV, D), (x @ wv).view(n, HKV, D)
            s = torch.einsum("ihgd,jhd->hgij", q, k) * D ** -0.5
            p = torch.softmax(s.masked_fill(~mask, -float("inf")), -1)
            x = x + torch.tanh(torch.einsum("hgij,jhd->ihgd", p, v).reshape(n, HIDDEN) @ wo)
        return self.head(x[-1])


def draw(logits, u, T, k, p):
    """One token, plainly; None where the uniform is near a border."""
    x = logits.double()
    if T == 0:
        return int(x.argmax())
    w = torch.exp((x - x.max()) / T)
    order = torch.argsort(-x, stable=True)
    mass = w[order][:k].cumsum(0)
    keep = order[:int((mass < p * mass[-1]).sum()) + 1].sort()[0]
    mass = w[keep].cumsum(0) / w[keep].sum()
    assert (mass - u).abs().min() > 1e-4
    return int(keep[int((mass <= u).sum())])


class Server:
    """Caches, staging and buffers of a step of fixed shape; in place, so that it can be captured."""

    def __init__(self, model, quantized, T=0.0, k=0, p=1.0, uniforms=None, workspace=None):
        self.m, self.quantized, self.settings, self.ws = model, quantized, (T, k, p), workspace
        E, P = HKV * D, 2 * LAYERS
        self.staging = torch.zeros((P, B, N, HKV, D), dtype=F32, device=DEV)
        if quantized:
            self.codes = torch.zeros((P, B, L, HKV, D), dtype=torch.uint8, device=DEV).view(F8)
            self.scales = torch.zeros((P, B, L, -(-E // 128)), dtype=torch.uint8, device=DEV).view(E8)
        else:
            self.cache = torch.full((P, B, L, HKV, D), float("nan"), dtype=F32, device=DEV)
        self.len = torch.zeros(B, dtype=I32, device=DEV)
        self.tokens = torch.zeros((B, N), dtype=I32, device=DEV)
        self.parents = torch.full((B, N), -2, dtype=I32, device=DEV)
        self.depth = torch.zeros((B, N), dtype=torch.long, device=DEV)
        self.uniforms = torch.zeros((B, L + N), device=DEV) if uniforms is None else uniforms.to(DEV)

    def step(self, sampled=None):
        """sampled: tokens given in place of drawn ones (a prompt's)."""
        at = self.len[:, None].long() + self.depth
        x = self.m.embed[self.tokens.long()] + self.m.place[at]
        for i, (wq, wk, wv, wo) in enumerate(self.m.layers):
            q = (x @ wq).view(B, N, HQ, D)
            self.staging[2 * i] = (x @ wk).view(B, N, HKV, D)
            self.staging[2 * i + 1] = (x @ wv).view(B, N, HKV, D)
            new = self.staging[2 * i], self.staging[2 * i + 1]
            if self.quantized:
                y = sv().spec_tree_attention_quantized(q, self.codes[2 * i], self.scales[2 * i], self.codes[2 * i + 1],
                                                       self.scales[2 * i + 1], *new, self.parents, self.len,
                                                       workspace=self.ws)
            else:
                y = sv().spec_tree_attention(q, self.cache[2 * i], self.cache[2 * i + 1], *new, self.parents, self.len,
                                             workspace=self.ws)
            x = x + torch.tanh(y.view(B, N, HIDDEN) @ wo)
        self.logits = self.m.head(x)
        T, k, p = self.settings
        if sampled is None:
            sampled = sv().spec_sample_tokens(self.logits, self.uniforms.gather(1, at), T, top_k=k, top_p=p)
        if self.quantized:
            return sv().spec_tree_commit_quantized(self.codes, self.scales, self.staging, self.tokens, self.parents,
                                                   sampled, self.len)
        return sv().spec_tree_commit(self.cache, self.staging, self.tokens, self.parents, sampled, self.len)

    def put(self, tokens, parents):
        """A tree per sequence: lists of tokens and parents, padded with absent nodes."""
        t, p, d = torch.zeros(B, N, dtype=I32), torch.full((B, N), -2, dtype=I32), torch.zeros(B, N, dtype=torch.long)
        for b in range(B):
            n = len(tokens[b])
            t[b, :n], p[b, :n] = torch.tensor(tokens[b], dtype=I32), torch.tensor(parents[b], dtype=I32)
            for i in range(1, n):
                d[b, i] = d[b, parents[b][i]] + 1
        self.tokens.copy_(t)
        self.parents.copy_(p)
        self.depth.copy_(d)


def drafts(g, right):
    """A tree behind a root: `right` (what will be emitted) along one branch up to a random depth, with wrong siblings."""
    tokens, parents, at = [], [], 0
    good = int(torch.randint(0, 5, (1,), generator=g))
    for i in range(1, N):
        up = at if len(right) and good > 0 and torch.rand((), generator=g) < 0.6 else \
            int(torch.randint(0, i, (1,), generator=g))
        if up == at and right and good > 0:
            tokens.append(right.pop(0))
            at, good = i, good - 1
        else:
            tokens.append(int(torch.randint(0, V, (1,), generator=g)))
        parents.append(up)
    return tokens, parents


def generate(server, prompts, want, steps, seed, run=None):
    """Emitted tokens of each sequence after its prompt; drafts come in part from `want`."""
    g = torch.Generator().manual_seed(seed)
    run = run or server.step
    got = [[] for _ in range(B)]
    # The prompt, as chains of up to N nodes whose drafts are taken as drawn.
    fed = [p[:-1] for p in prompts]
    server.put([f for f in fed], [[i - 1 for i in range(len(f))] for f in fed])
    kept = server.settings
    sampled = torch.full((B, N), V + 1, dtype=I32)
    for b, f in enumerate(fed):
        sampled[b, :max(0, len(f) - 1)] = torch.tensor(f[1:], dtype=I32)
    server.step(sampled.to(DEV))
    assert server.len.tolist() == [len(f) for f in fed]
    roots, more, taken = [p[-1] for p in prompts], 0, []
    for _ in range(steps):
        trees = [drafts(g, list(want[b][len(got[b]):])) for b in range(B)]
        server.put([[roots[b]] + trees[b][0] for b in range(B)], [[-1] + trees[b][1] for b in range(B)])
        acc, out, path, status = run()
        assert status.tolist() == [0] * B
        for b in range(B):
            new = [t for t in out[b].tolist() if t >= 0]
            assert len(new) == acc[b].item() + 1
            got[b] += new
            roots[b] = new[-1]
            taken.append(len(new))
    assert server.settings == kept
    return got, taken


@pytest.fixture(scope="module")
def model():
    return Model()


@pytest.fixture(scope="module")
def gpu_model(model):
    return model.to(F32, DEV)


PROMPTS = [[3, 14, 15, 9], [26], [5, 35], [8, 9, 7, 9, 3, 2, 3, 8, 4]]


def plain_run(model, T, k, p, u, count):
    """What the model emits without drafts."""
    out = []
    for b, prompt_ in enumerate(PROMPTS):
        seq = list(prompt_)
        for _ in range(count):
            seq.append(draw(model.plain(seq), float(u[b, len(seq) - 1]), T, k or V, p))
        out.append(seq[len(prompt_):])
    return out


def uniforms(seed):
    return torch.rand((B, L + N), generator=torch.Generator().manual_seed(seed)) * 0.98 + 0.01


@pytest.mark.parametrize("T,k,p", [(0.0, 0, 1.0), (0.8, 0, 1.0), (1.0, 10, 0.9)])
def test_trees_emit_what_the_model_emits_without_drafts(model, gpu_model, T, k, p):
    """The n-th token of a sequence is drawn with its n-th uniform, in a tree as without: the same tokens."""
    count = 40
    for seed in range(2, 40):   # uniforms that are far from every border of the plain run
        u = uniforms(seed)
        try:
            want = plain_run(model, T, k, p, u, count)
            break
        except AssertionError:
            continue
    got, taken = generate(Server(gpu_model, False, T, k, p, u), PROMPTS, want, 9, 1)
    for b in range(B):
        n = min(len(got[b]), count)
        assert n >= 9 and got[b][:n] == want[b][:n], b
    assert max(taken) > 2 and min(taken) >= 1   # drafts were accepted, and were not


def reads(server):
    """The cache's values in fp32, as far as they are committed."""
    E = HKV * D
    out = torch.zeros((2 * LAYERS, B, L, HKV, D), dtype=F32, device=DEV)
    if server.quantized:
        sv().spec_kv_read_quantized(server.codes, server.scales, server.len, out)
    else:
        for b, n in enumerate(server.len.tolist()):
            out[:, b, :n] = server.cache[:, b, :n]
    return out


def test_the_8_bit_cache_holds_the_committed_entries_rounded(gpu_model):
    """The same drafts and draws over both caches for a step: the committed entries are each other's, in 8 bits."""
    a, b = Server(gpu_model, False), Server(gpu_model, True)
    for s in (a, b):
        s.put([p[:N] for p in PROMPTS], [[i - 1 for i in range(len(p))] for p in PROMPTS])
        sampled = torch.full((B, N), V + 1, dtype=I32)
        for i, f in enumerate(PROMPTS):
            sampled[i, :len(f) - 1] = torch.tensor(f[1:], dtype=I32)
        s.step(sampled.to(DEV))
    assert a.len.tolist() == b.len.tolist() == [len(p) for p in PROMPTS]
    x, y = reads(a), reads(b)
    # e4m3 with a block's scale: half a step of 2^-4, or of the smallest code 2^-9 at the scale of the block's largest
    rows = x.flatten(-2).abs().amax(-1)[..., None, None]
    assert ((x - y).abs() <= 2.0 ** -4 * x.abs() + rows * 2.0 ** -9).all()
    # and attention reads those values: over the 8-bit cache as over the values read back
    q = torch.randn((B, N, HQ, D), generator=torch.Generator().manual_seed(3)).to(DEV)
    t = (b.staging[0], b.staging[1], b.parents, b.len)
    got = sv().spec_tree_attention_quantized(q, b.codes[0], b.scales[0], b.codes[1], b.scales[1], *t)
    want = sv().spec_tree_attention(q, y[0], y[1], *t)
    assert (got - want).abs().max() < 1e-5


@pytest.mark.parametrize("quantized", [False, True])
def test_a_captured_step_is_the_eager_one(gpu_model, quantized):
    """One capture, replayed for every step of a generation with eager work between; default and own workspaces."""
    u = uniforms(7)
    eager, _ = generate(Server(gpu_model, quantized, 0.9, 20, 0.95, u), PROMPTS, [[], [], [], []], 6, 2)
    for workspace in (None, sv().Workspace(DEV)):
        s = Server(gpu_model, quantized, 0.9, 20, 0.95, u, workspace)
        held = {}

        def run():
            if "graph" not in held:
                kept = [t.clone() for t in ((s.codes, s.scales) if quantized else (s.cache,))] + [s.len.clone()]
                side = torch.cuda.Stream()
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    s.step()
                torch.cuda.current_stream().wait_stream(side)
                held["graph"] = torch.cuda.CUDAGraph()
                with torch.cuda.graph(held["graph"]):
                    held["out"] = s.step()
                for t, k in zip(((s.codes, s.scales) if quantized else (s.cache,)) + (s.len,), kept):
                    t.copy_(k)
            held["graph"].replay()
            torch.cuda.synchronize()
            sv().spec_sample_tokens(s.logits, torch.zeros((B, N), device=DEV), 1.0, top_p=0.5)
            return held["out"]
        got, _ = generate(s, PROMPTS, [[], [], [], []], 6, 2, run)
        assert got == eager


def long_inputs(seed, quantized):
    g = torch.Generator(DEV).manual_seed(seed)
    q = torch.randn((1, 5, 8, 128), generator=g, device=DEV).to(BF)
    new = torch.randn((2, 1, 5, 1, 128), generator=g, device=DEV).to(BF)
    par = torch.tensor([[-1, 0, 0, 1, 2]], dtype=I32, device=DEV)
    n = torch.tensor([9000 - seed], dtype=I32, device=DEV)
    if quantized:
        codes = torch.randint(0, 120, (2, 1, 9000, 1, 128), generator=g, device=DEV, dtype=torch.uint8).view(F8)
        scales = torch.full((2, 1, 9000, 1), 120, dtype=torch.uint8, device=DEV).view(E8)
        return lambda **k: sv().spec_tree_attention_quantized(q, codes[0], scales[0], codes[1], scales[1], new[0],
                                                              new[1], par, n, **k)
    cache = torch.randn((2, 1, 9000, 1, 128), generator=g, device=DEV).to(BF)
    return lambda **k: sv().spec_tree_attention(q, cache[0], cache[1], new[0], new[1], par, n, **k)


@pytest.mark.parametrize("quantized", [False, True])
def test_calls_in_splits_on_several_streams_and_graphs_at_once(quantized):
    """Default workspaces: calls on three streams, two graphs captured on one stream and replayed on two, and eager calls
    on the stream they were captured on."""
    fs = [long_inputs(i, quantized) for i in range(3)]
    want = [f() for f in fs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(20):
        for f, s in zip(fs, streams):
            with torch.cuda.stream(s):
                got.append(f())
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 3]) for i, g in enumerate(got))
    graphs, outs = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=streams[2]):
            outs.append(fs[i]())
    for _ in range(10):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            last = fs[2]()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(last, want[2])


def test_calls_on_an_explicit_stream(gpu_model):
    """Results on another stream than the current one, for every operator of the step."""
    s = torch.cuda.Stream()
    f = long_inputs(1, False)
    want = f()
    x = torch.randn((300, 5000), generator=torch.Generator(DEV).manual_seed(2), device=DEV)
    u = torch.rand((300,), generator=torch.Generator(DEV).manual_seed(3), device=DEV)
    tokens = sv().spec_sample_tokens(x, u, 1.0, top_k=40)
    torch.cuda.synchronize()
    got, again = f(stream=s), sv().spec_sample_tokens(x, u, 1.0, top_k=40, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want) and torch.equal(again, tokens)


def test_calls_from_threads_on_one_stream():
    fs = [long_inputs(i, False) for i in range(4)]
    want = [f() for f in fs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        for _ in range(25):
            got = fs[i]()
            torch.cuda.current_stream().synchronize()
            if not torch.equal(got, want[i]):
                bad.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad

"""Windowed attention with sinks on the GPU, against softmax over the visible keys in 64 bits.

Everything that no query may see is poisoned: the pool starts as NaN and only visible keys are written, hidden blocks'
table entries are out of range.

Tolerance of an output o = sum w_t v_t, with A = sum w_t |v_t|: the weights are rounded to the products' 16-bit type
(half a step u of each: u A), the output to its own (u |o|), the scores' 32-bit sums of d products and the exponentials
are off by less than 2^-13 each way (2^-12 A; CUDA cores, f32: 2^-15 A), and each of the K weights in binary16 by half
its smallest step (K 2^-25 max |v|)."""
import math

import pytest
import torch

import paged_kv_cache_80_gb300 as pkv

pytestmark = pytest.mark.gpu

ACT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.bfloat16}
SCALES = (0.03125, 0.0625)
POISON_ID = (1 << 30, -1)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


class Batch:
    """Sequences of given lengths whose last `chunks` tokens are queries, poisoned where no query sees."""

    def __init__(self, dtype, lens, window, n_sink, chunks=None, H_q=16, H_kv=2, d=128, B=16, L=1, layer=0, seed=0,
                 q_scale=1.0, extra_rows=0, blocks=None, min_block=0):
        self.dtype, self.lens, self.window, self.n_sink, self.layer = dtype, lens, window, n_sink, layer
        self.H_q, self.H_kv, self.d, self.B, self.G = H_q, H_kv, d, B, H_q // H_kv
        self.decode = chunks is None
        self.chunks = [1] * len(lens) if chunks is None else chunks
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 3)
        rnd = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
        need = [-(-n // B) for n in lens]
        self.W = max(need + [1]) + 1
        self.blocks = sum(need) + 5 if blocks is None else blocks
        order = (torch.randperm(self.blocks - min_block, generator=g, device="cuda") + min_block).tolist()
        self.pool = pkv.pkv_pool_create(L, H_q, H_kv, d, B, dtype, self.blocks)
        shape = (self.blocks, L, H_kv, B, d)
        if dtype == "e4m3":
            pkv.pkv_pool_set_kv_scales(self.pool, *SCALES)
            self.kp, self.vp = (torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
        else:
            self.kp, self.vp = (torch.full(shape, math.nan, dtype=ACT[dtype], device="cuda") for _ in range(2))
        self.tables = torch.tensor([[POISON_ID[(i + l) % 2] for l in range(self.W)] for i in range(len(lens))],
                                   dtype=torch.int32).reshape(len(lens), self.W)
        self.data = []
        for i, (n, c) in enumerate(zip(lens, self.chunks)):
            first = max(0, n - c + 1 - window)
            t = torch.arange(n, device="cuda")
            t = t[(t < n_sink) | (t >= first)] if c else t[:0]
            k, v = rnd(len(t), H_kv, d), rnd(len(t), H_kv, d)
            if dtype == "e4m3":
                k, v = ((x / s).clamp(-448, 448).to(torch.float8_e4m3fn) for x, s in zip((k, v), SCALES))
                stored, k, v = (k.view(torch.uint8), v.view(torch.uint8)), k.double() * SCALES[0], v.double() * SCALES[1]
            else:
                stored = k.to(ACT[dtype]), v.to(ACT[dtype])
                k, v = stored[0].double(), stored[1].double()
            for b in sorted(set((t // B).tolist())):
                self.tables[i, b] = order.pop()
            at = self.tables[i].cuda().long()[t // B]
            self.kp[at, layer, :, t % B], self.vp[at, layer, :, t % B] = stored
            self.data.append((t, k, v))
        offs = [0]
        for c in self.chunks if not self.decode else [1] * len(lens):
            offs.append(offs[-1] + c)
        self.offs = offs
        self.tables = self.tables.cuda()
        self.lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.offs_d = torch.tensor(offs, dtype=torch.int32, device="cuda")
        rows = offs[-1] + extra_rows
        self.q = (rnd(rows, H_q, d) * q_scale).to(ACT[dtype])
        self.out = torch.full((rows, H_q, d), math.nan, dtype=ACT[dtype], device="cuda")
        self.scale = 1.0 / math.sqrt(d)
        self.ws = torch.empty(pkv.pkv_decode_workspace_size(self.pool, len(lens)), dtype=torch.uint8, device="cuda")

    def call(self, max_q=None, **kw):
        a = dict(q=self.q, kp=self.kp, vp=self.vp, tables=self.tables, lens=self.lens_d, window=self.window,
                 n_sink=self.n_sink, scale=self.scale, out=self.out, ws=self.ws, offs=self.offs_d)
        a.update(kw)
        if self.decode:
            pkv.pkv_decode_attention_window(self.pool, self.layer, a["q"], a["kp"], a["vp"], a["tables"], a["lens"],
                                            a["window"], a["n_sink"], a["scale"], a["out"], a["ws"])
        else:
            pkv.pkv_prefill_attention_window(self.pool, self.layer, a["q"], a["offs"],
                                             max(self.chunks) if max_q is None else max_q, a["kp"], a["vp"], a["tables"],
                                             a["lens"], a["window"], a["n_sink"], a["scale"], a["out"])

    def check(self, only=None):
        pkv.pkv_check_device_error()
        t16 = torch.float16 if self.dtype in ("f16", "e4m3") else torch.bfloat16
        for i, (n, c) in enumerate(zip(self.lens, self.chunks)):
            if only is not None and i not in only:
                continue
            rows = slice(self.offs[i], self.offs[i] + c)
            got = self.out[rows].double()
            if n == 0:
                assert bool((got == 0).all())
                continue
            if c == 0:
                continue
            t, k, v = self.data[i]
            p = torch.arange(n - c, n, device="cuda")[:, None]
            seen = (t <= p) & ((t > p - self.window) | (t < self.n_sink))  # [c, K]
            q = self.q[rows].double().unflatten(1, (self.H_kv, self.G))
            z = torch.einsum("chgd,thd->hgct", q, k) * self.scale
            z = z.masked_fill(~seen, -math.inf)
            w = (z - torch.logsumexp(z, -1, keepdim=True)).exp()
            ref = torch.einsum("hgct,thd->chgd", w, v).flatten(1, 2)
            A = torch.einsum("hgct,thd->chgd", w, v.abs()).flatten(1, 2)
            if self.dtype == "f32":
                tol = A * 2.0**-15
            else:
                tol = A * (half_step(t16) + 2.0**-12) + ref.abs() * half_step(ACT[self.dtype])
                if t16 is torch.float16:
                    tol = tol + len(t) * 2.0**-25 * v.abs().max()
            assert bool(torch.isfinite(got).all()), f"sequence {i}"
            worst = float(((got - ref).abs() / tol).max())
            assert worst <= 1.0, f"sequence {i} of length {n}: {worst:.3f} of the tolerance"
        if only is None:  # rows behind the last sequence
            assert bool(torch.isnan(self.out[self.offs[-1]:]).all())


LENS = [0, 1, 15, 16, 17, 33, 100, 129, 130, 500, 1999]
WINDOWS = [(1, 0), (1, 1), (16, 4), (33, 17), (128, 0), (129, 200), (1000, 64), (2**31 - 1, 2**31 - 1), (64, 2**31 - 1)]


@pytest.mark.parametrize("window,n_sink", WINDOWS)
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_decode_windows(dtype, window, n_sink):
    b = Batch(dtype, LENS, window, n_sink)
    b.call()
    b.check()


@pytest.mark.parametrize("kw", [
    dict(dtype="f16", H_q=64, H_kv=8), dict(dtype="bf16", H_q=4, H_kv=4, d=64, B=32), dict(dtype="f16", H_q=7, H_kv=1, d=64),
    dict(dtype="bf16", H_q=32, H_kv=2), dict(dtype="f16", H_q=24, H_kv=2, d=64, B=48), dict(dtype="e4m3", H_q=32, H_kv=2, B=64),
    dict(dtype="bf16", H_q=16, H_kv=2, L=3, layer=2),
    # CUDA cores: f32, head sizes and block sizes that are not the tensor cores'
    dict(dtype="f32", H_q=12, H_kv=12, d=64), dict(dtype="f32", H_q=16, H_kv=2, d=256, B=7), dict(dtype="bf16", H_q=8, H_kv=2, d=96),
    dict(dtype="f16", H_q=32, H_kv=2, d=34, B=5), dict(dtype="e4m3", H_q=4, H_kv=1, d=72), dict(dtype="bf16", H_q=8, H_kv=1, B=24),
], ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
@pytest.mark.parametrize("window,n_sink", [(50, 4), (333, 0), (7, 40)])
def test_decode_geometries(kw, window, n_sink):
    b = Batch(lens=LENS, window=window, n_sink=n_sink, **kw)
    b.call()
    b.check()


# more (sequence, KV head) pairs than SMs: the persistent kernel, whose warps cut pairs anywhere
MANY = [(i * 131) % 2100 for i in range(60)] + [0, 1, 16, 17]


@pytest.mark.parametrize("kw", [
    dict(dtype="bf16", H_q=64, H_kv=8), dict(dtype="f16", H_q=8, H_kv=8, d=64, B=32), dict(dtype="f16", H_q=64, H_kv=4, d=64),
    dict(dtype="bf16", H_q=96, H_kv=8, B=48), dict(dtype="e4m3", H_q=28, H_kv=4, B=64), dict(dtype="e4m3", H_q=128, H_kv=8),
], ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
@pytest.mark.parametrize("window,n_sink", [(1, 0), (50, 4), (333, 0), (129, 200), (7, 40), (2**31 - 1, 5)])
def test_decode_many_pairs(kw, window, n_sink):
    b = Batch(lens=MANY, window=window, n_sink=n_sink, **kw)
    b.call()
    b.check()


def test_decode_many_pairs_replayed():
    """The persistent kernel counts the parts of a pair anew at every replay."""
    a = Batch("bf16", MANY, 900, 4, H_q=64, H_kv=8)
    b = Batch("e4m3", MANY[::-1], 500, 0, H_q=32, H_kv=4, seed=1)
    ws = a.ws if a.ws.numel() >= b.ws.numel() else b.ws
    graphs = []
    for x in (a, b):
        x.call(ws=ws)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            x.call(ws=ws)
    for turn in range(3):
        for x, graph in zip((a, b), graphs):
            x.q.copy_(torch.randn_like(x.q))
            x.out.fill_(math.nan)
            graph.replay()
            x.check()
    plain = torch.cuda.CUDAGraph()  # the call without a window, too
    whole = Batch("bf16", MANY, 4096, 0, H_q=64, H_kv=8)
    pkv.pkv_decode_attention(whole.pool, 0, whole.q, whole.kp, whole.vp, whole.tables, whole.lens_d, whole.scale, whole.out, whole.ws)
    with torch.cuda.graph(plain):
        pkv.pkv_decode_attention(whole.pool, 0, whole.q, whole.kp, whole.vp, whole.tables, whole.lens_d, whole.scale, whole.out,
                                 whole.ws)
    for _ in range(3):
        whole.q.copy_(torch.randn_like(whole.q))
        whole.out.fill_(math.nan)
        plain.replay()
        whole.check()


def test_decode_one_long_sequence_over_the_whole_grid():
    b = Batch("bf16", [70001], 20011, 5, H_q=64, H_kv=8)
    b.call()
    b.check()


def test_decode_more_sequences_than_the_kernel_plans_itself():
    lens = [(i * 37) % 300 for i in range(4100)]
    b = Batch("bf16", lens, 40, 3, H_q=8, H_kv=1, d=64)
    b.call()
    b.check(only=set(range(0, 4100, 61)) | {4099})


def test_decode_sharp_scores():
    """Scores up to hundreds: the running maximum moves, most weights vanish."""
    b = Batch("f16", [900, 77, 2000], 700, 9, q_scale=30.0)
    b.call()
    pkv.pkv_check_device_error()
    assert bool(torch.isfinite(b.out).all())
    f = Batch("f32", [900, 77, 2000], 700, 9, q_scale=30.0, d=64)
    f.call()
    # 30 times the score, and its 32-bit error with it: 30 * 2^-15 A
    f.out, keep = f.out.clone(), f.out
    for i in range(3):
        t, k, v = f.data[i]
        z = torch.einsum("hgd,thd->hgt", f.q[i].double().unflatten(0, (f.H_kv, f.G)), k) * f.scale
        w = (z - torch.logsumexp(z, -1, keepdim=True)).exp()
        ref, A = (torch.einsum("hgt,thd->hgd", w, x).flatten(0, 1) for x in (v, v.abs()))
        assert bool(((keep[i].double() - ref).abs() <= 30 * 2.0**-15 * A).all())


CHUNKS = [
    ([0, 1, 16, 65, 300, 700, 1300], [0, 1, 16, 33, 64, 500, 1]),
    ([257, 2000, 129], [257, 600, 128]),
]


@pytest.mark.parametrize("lens,chunks", CHUNKS)
@pytest.mark.parametrize("window,n_sink", WINDOWS)
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_prefill_windows(dtype, window, n_sink, lens, chunks):
    b = Batch(dtype, lens, window, n_sink, chunks, extra_rows=3)
    b.call()
    b.check()


@pytest.mark.parametrize("kw", [
    dict(dtype="f16", H_q=64, H_kv=8), dict(dtype="bf16", H_q=4, H_kv=4, B=32), dict(dtype="bf16", H_q=6, H_kv=2, B=64),
    dict(dtype="f16", H_q=12, H_kv=1), dict(dtype="bf16", H_q=64, H_kv=1), dict(dtype="e4m3", H_q=32, H_kv=2, B=128),
    dict(dtype="e4m3", H_q=5, H_kv=5), dict(dtype="bf16", H_q=128, H_kv=1), dict(dtype="e4m3", H_q=100, H_kv=1),
    dict(dtype="f16", H_q=66, H_kv=1, d=64), dict(dtype="bf16", H_q=16, H_kv=2, L=2, layer=1),
    # mma.sync (d_head 64)
    dict(dtype="bf16", H_q=16, H_kv=2, d=64), dict(dtype="f16", H_q=3, H_kv=3, d=64, B=32), dict(dtype="f16", H_q=7, H_kv=1, d=64),
    # CUDA cores
    dict(dtype="f32", H_q=12, H_kv=12, d=64), dict(dtype="bf16", H_q=16, H_kv=2, d=96, B=9), dict(dtype="e4m3", H_q=8, H_kv=2, d=40),
], ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
@pytest.mark.parametrize("window,n_sink", [(50, 4), (333, 0), (7, 70)])
def test_prefill_geometries(kw, window, n_sink):
    b = Batch(lens=[40, 500, 900, 131], window=window, n_sink=n_sink, chunks=[40, 200, 3, 130], **kw)
    b.call()
    b.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_prefill_a_whole_long_prompt(dtype):
    b = Batch(dtype, [9000], 900, 20, [9000], H_q=8, H_kv=1)
    b.call()
    b.check()


def test_prefill_behind_a_history_longer_than_the_staged_table():
    b = Batch("bf16", [70001], 3001, 5, [40], H_q=8, H_kv=1)
    b.call()
    b.check()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("e4m3", 128), ("f16", 64)])
@pytest.mark.parametrize("n", [130, 700])
def test_prefill_many_sequences(dtype, d, n):
    """More sequences than the kernel's table has entries, many without a chunk."""
    chunks = [(i * 7) % 45 if i % 3 else 0 for i in range(n)]
    lens = [c + (i * 13) % 60 for i, c in enumerate(chunks)]
    b = Batch(dtype, lens, 31, 3, chunks, H_q=8, H_kv=1, d=d)
    b.call()
    b.check(only=set(range(0, n, 19)) | set(range(n - 6, n)))


def test_prefill_without_a_chunk_and_two_streams_at_once():
    b = Batch("bf16", [20, 30], 16, 2, [0, 0], extra_rows=4)
    b.call(max_q=8)
    b.check()
    many = [Batch(t, [600, 900, 33], 200, 4, c, seed=i) for i, (t, c) in
            enumerate([("bf16", [600, 300, 33]), ("e4m3", [600, 900, 1]), ("bf16", None), ("e4m3", None)])]
    streams = [torch.cuda.Stream() for _ in many]
    torch.cuda.synchronize()
    for _ in range(3):
        for x, s in zip(many, streams):
            with torch.cuda.stream(s):
                x.call()
    torch.cuda.synchronize()
    for x in many:
        x.check()


@pytest.mark.parametrize("chunks", [None, [40, 1]])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 96)])
def test_offsets_past_32_bits(dtype, d, chunks):
    """Blocks at the far end of a pool of more than 2^31 elements."""
    H_kv, B = 8, 16
    blocks = 2**31 // (H_kv * d * B) + 80
    b = Batch(dtype, [300, 41], 100, 4, chunks, H_q=16, H_kv=H_kv, d=d, B=B, blocks=blocks, min_block=blocks - 60)
    b.call()
    b.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_a_wide_window_is_the_whole_sequence(dtype):
    """window >= len: the keys of the calls without a window.  The two may cut a sequence in different places, so that
    their partial sums are rounded differently: each is held to the definition, not to the other's bits."""
    b = Batch(dtype, LENS, 4096, 0)
    b.call()
    b.check()
    pkv.pkv_decode_attention(b.pool, 0, b.q, b.kp, b.vp, b.tables, b.lens_d, b.scale, b.out.fill_(math.nan), b.ws)
    b.check()
    p = Batch(dtype, [300, 700], 4096, 0, [300, 77])
    p.call()
    p.check()
    pkv.pkv_prefill_attention(p.pool, 0, p.q, p.offs_d, 300, p.kp, p.vp, p.tables, p.lens_d, p.scale, p.out.fill_(math.nan))
    p.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("H_q,H_kv", [(3, 1), (24, 1), (80, 2)])  # 128 is no multiple of the queries of a KV head
def test_prefill_rows_depend_on_their_own_sequence_alone(dtype, H_q, H_kv):
    """The same bits whatever the next sequence's queries, the rows behind the last one and the calls before."""
    b = Batch(dtype, [700, 300, 90], 200, 4, [33, 130, 7], H_q=H_q, H_kv=H_kv, extra_rows=9)
    b.call()
    b.check()
    first = b.out.clone()
    rows = slice(b.offs[1], b.offs[2])
    others = [i for i in range(b.offs[-1]) if not b.offs[1] <= i < b.offs[2]]
    q = b.q.clone()
    for k in (100.0, 0.0, 30.0):
        b.q[others] = q[others] * k
        b.q[b.offs[-1]:] = math.nan if k else 1000.0
        b.call()
        assert torch.equal(b.out[rows], first[rows]), k
    b.q.copy_(q)
    b.call()
    assert torch.equal(b.out[:b.offs[-1]], first[:b.offs[-1]])


@pytest.mark.parametrize("chunks", [None, [5, 1, 40]])
def test_windows_past_32_bits_are_every_key(chunks):
    b = Batch("bf16", [300, 1, 40], 2**31 - 1, 0, chunks)
    for kw in (dict(window=2**32 + 5), dict(window=2**31), dict(window=3, n_sink=2**32 + 1)):
        b.out.fill_(math.nan)
        b.call(**kw)
        b.check()


def test_replayed_graphs_that_share_a_workspace():
    """Every replay counts its split pairs anew: two graphs, replayed in turn with new lengths, queries and workspace bytes."""
    a = Batch("bf16", [3000, 17, 800], 900, 4, H_q=64, H_kv=8)
    b = Batch("bf16", [5000], 4000, 0, H_q=64, H_kv=8, seed=1)
    ws = a.ws if a.ws.numel() >= b.ws.numel() else b.ws
    for x in (a, b):
        x.call(ws=ws)
        x.check()
    graphs = []
    for x in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            x.call(ws=ws)
        graphs.append(graph)
    for turn in range(3):
        for x, graph in zip((a, b), graphs):
            x.q.copy_(torch.randn_like(x.q))
            x.out.fill_(math.nan)
            graph.replay()
            x.check()
        if turn == 1:
            ws.random_(0, 256)
    p = Batch("bf16", [300, 900], 129, 4, [300, 200])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.call()
    for _ in range(2):
        p.q.copy_(torch.randn_like(p.q))
        p.out.fill_(math.nan)
        graph.replay()
        p.check()


def test_another_stream():
    side = torch.cuda.Stream()
    for b in (Batch("bf16", LENS, 100, 4), Batch("bf16", [300, 900], 129, 4, [300, 200])):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            b.call()
        side.synchronize()
        b.check()


@pytest.mark.parametrize("d", [128, 64, 96])
def test_bad_values_are_recorded(d):
    """A length past the table, a visible block out of range and chunks outside q: the error word, and no other sequence hurt."""

    def recorded(code):
        with pytest.raises(pkv.PkvError) as e:
            pkv.pkv_check_device_error()
        assert f"code {code}" in str(e.value)

    b = Batch("bf16", [100, 50, 200], 60, 4, d=d)
    b.tables[1, 2] = b.blocks  # holds the newest keys of sequence 1
    b.call()
    recorded(3)
    b.check(only={0, 2})
    b = Batch("bf16", [100, 50, 200], 60, 4, d=d)
    b.lens_d[0] = -5
    b.call()
    recorded(2)
    b.check(only={1, 2})
    assert bool((b.out[0] == 0).all())
    p = Batch("bf16", [100, 50, 200], 60, 4, [30, 50, 7], d=d)
    p.lens_d[1] = p.W * p.B + 1
    p.call()
    recorded(2)
    p.check(only={0, 2})
    if d != 96:  # the CUDA-core kernel goes by rows and needs no bound
        p = Batch("bf16", [300, 50], 60, 4, [300, 50], d=d)
        p.call(max_q=50)
        recorded(6)
        p.check(only={1})
        p = Batch("bf16", [300, 50], 60, 4, [300, 50], d=d)
        p.offs_d[2] = 351
        p.call()
        recorded(6)
        p.check(only={0})


def test_refusals():
    b = Batch("bf16", [100, 50], 60, 4)
    p = Batch("bf16", [100, 50], 60, 4, [3, 50])
    for x in (b, p):
        for kw, text in [(dict(window=0), "window"), (dict(window=-1), "window"), (dict(n_sink=-1), "n_sink"),
                         (dict(scale=0.0), "scale"), (dict(scale=-1.0), "scale"), (dict(scale=math.nan), "scale")]:
            with pytest.raises(pkv.PkvError, match=text):
                x.call(**kw)
        for kw, error, text in [(dict(q=x.q.float()), TypeError, "q is"), (dict(out=x.out[:1]), ValueError, "out"),
                                (dict(kp=x.kp[:-1]), ValueError, "k_pool"), (dict(vp=x.vp.half()), TypeError, "v_pool"),
                                (dict(tables=x.tables[:1]), ValueError, "block_tables"), (dict(lens=x.lens_d.long()), TypeError, "seq_lens"),
                                (dict(tables=x.tables[:, ::2]), ValueError, "contiguous")]:
            with pytest.raises(error, match=text):
                x.call(**kw)
        assert bool(torch.isnan(x.out).all())
        for name, text in [("q", "q must"), ("tables", "block_tables must"), ("lens", "seq_lens must"), ("out", "out must")]:
            for wrong in (None, [1, 2], getattr(x, {"lens": "lens_d"}.get(name, name)).cpu()):
                with pytest.raises(TypeError, match=text):
                    x.call(**{name: wrong})
        shifted = torch.zeros(x.q.numel() + 1, dtype=x.q.dtype, device="cuda")[1:].view(x.q.shape)
        for name in ("q", "out"):
            with pytest.raises(pkv.PkvError, match="aligned"):
                x.call(**{name: shifted})
    for wrong in (None, b.ws.cpu()):
        with pytest.raises(TypeError, match="workspace must"):
            b.call(ws=wrong)
    with pytest.raises(pkv.PkvError, match="workspace"):
        b.call(ws=b.ws[:256])
    with pytest.raises(ValueError, match="q_offsets"):
        p.call(offs=p.offs_d[:-1])
    with pytest.raises(pkv.PkvError, match="max_q"):
        p.call(max_q=0)
    wide = Batch("f32", [20], 8, 0, H_q=32, H_kv=1, d=64)
    with pytest.raises(pkv.PkvError, match="16 query heads"):
        wide.call()
    with pytest.raises(pkv.PkvError, match="16 query heads"):
        Batch("f32", [20], 8, 0, [20], H_q=32, H_kv=1, d=64).call()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_prompt_and_steps_with_rotary_append(dtype):
    """As a model's layer uses them: two prompt chunks, then decode steps, the cache filled by the rotary append and the
    blocks planned by the pool; every attention is checked against the cache's own contents."""
    H_q, H_kv, d, B, window, n_sink = 16, 2, 128, 16, 48, 4
    pool = pkv.pkv_pool_create(1, H_q, H_kv, d, B, dtype, 64)
    if dtype == "e4m3":
        pkv.pkv_pool_set_kv_scales(pool, *SCALES)
    store = torch.uint8 if dtype == "e4m3" else torch.bfloat16
    kp, vp = (torch.zeros((64, 1, H_kv, B, d), dtype=store, device="cuda") for _ in range(2))
    ids = [pkv.pkv_seq_create(pool) for _ in range(3)]
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    rotary = pkv.Rotary((1e4 ** (-torch.arange(d // 2, device="cuda") / (d // 2))).float())
    W, scale, lens = 16, d**-0.5, [0, 0, 0]
    for step, n_new in enumerate([[100, 33, 1], [17, 60, 40]] + [[1, 1, 1]] * 20):
        slots, cows = pkv.pkv_plan_append(pool, ids, n_new)
        assert len(cows) == 0
        n = sum(n_new)
        qkv = torch.randn((n, (H_q + 2 * H_kv) * d), generator=g, device="cuda").bfloat16()
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([H_q * d, H_kv * d, H_kv * d], 1))
        pos = torch.cat([torch.arange(l, l + c) for l, c in zip(lens, n_new)]).to(torch.int32).cuda()
        rotated = torch.empty((n, H_q, d), dtype=torch.bfloat16, device="cuda")
        pkv.pkv_append_kv_rotary(pool, 0, rotary, q, k, v, pos, torch.from_numpy(slots).cuda(), rotated, kp, vp)
        tables, seq_lens = pkv.pkv_export_tables(pool, ids, W)
        lens = seq_lens.tolist()
        b = Batch.__new__(Batch)
        b.dtype, b.lens, b.window, b.n_sink, b.layer, b.H_q, b.H_kv, b.d, b.B, b.G = dtype, lens, window, n_sink, 0, H_q, H_kv, d, B, H_q // H_kv
        b.decode, b.chunks, b.pool, b.kp, b.vp, b.W, b.scale = step >= 2, n_new, pool, kp, vp, W, scale
        b.tables, b.lens_d = torch.from_numpy(tables.copy()).cuda(), torch.from_numpy(seq_lens.copy()).cuda()
        b.offs = [0, n_new[0], n_new[0] + n_new[1], n]
        b.offs_d = torch.tensor(b.offs, dtype=torch.int32, device="cuda")
        b.q, b.out = rotated, torch.full_like(rotated, math.nan)
        b.ws = torch.empty(pkv.pkv_decode_workspace_size(pool, 3), dtype=torch.uint8, device="cuda")
        b.data = []
        for i, m in enumerate(lens):
            t = torch.arange(m, device="cuda")
            at = b.tables[i].long()[t // B]
            kk, vv = kp[at, 0, :, t % B], vp[at, 0, :, t % B]
            if dtype == "e4m3":
                kk, vv = kk.view(torch.float8_e4m3fn).double() * SCALES[0], vv.view(torch.float8_e4m3fn).double() * SCALES[1]
            b.data.append((t, kk.double(), vv.double()))
        b.call()
        b.check()
        w = pos.double()[:, None] * rotary.inv_freq.double()
        z = torch.polar(torch.ones_like(w), w)[:, None] * torch.complex(*q.double().chunk(2, -1))
        assert bool((rotated.double() - torch.cat([z.real, z.imag], -1)).abs().max() <= 2.0**-8 * 6 + 2.0**-17)

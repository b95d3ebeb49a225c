"""Append with rotary positions on the GPU, against the rotation in 64 bits and a plain write at the slots.

Tolerance of a rotated element y of a pair of radius r = |(x1, x2)|: half a step of its type, and what the 32-bit rotation
may be off: the angle by pi 2^-24 (rounding the phase to 24 bits) and 4.8e-7 more at positions near 2^31 (the 64-bit
turns), cosine and sine by 2 units of 2^-24 each, the two products and their sum by 3 -- r 2^-20 together for positions
below 2^20, r 2^-19 for any."""
import numpy as np
import pytest
import torch

import paged_kv_cache_80_gb300 as pkv

pytestmark = pytest.mark.gpu

ACT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.bfloat16}
STORE = dict(ACT, e4m3=torch.uint8)
SCALES = (0.03125, 0.09375)


class Case:
    """Inputs, the framework's call and the expected arrays of one append."""

    def __init__(self, dtype, n, H_q=8, H_kv=2, d=64, B=16, rot=None, interleaved=False, axes=None, L=1, layer=0, seed=0,
                 top=1 << 20, pad=0, blocks=None):
        self.dtype, self.n, self.H_q, self.H_kv, self.d, self.B, self.layer = dtype, n, H_q, H_kv, d, B, layer
        self.rot, self.interleaved = d if rot is None else rot, interleaved
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 17)
        self.blocks = n // B + n + 3 if blocks is None else blocks
        self.pool = pkv.pkv_pool_create(L, H_q, H_kv, d, B, dtype, self.blocks)
        if dtype == "e4m3":
            pkv.pkv_pool_set_kv_scales(self.pool, *SCALES)
        row = (H_q + 2 * H_kv) * d + pad  # one projection's row; pad shifts every later row's alignment
        self.qkv = torch.randn((n, row), generator=g, device="cuda").to(ACT[dtype])
        self.q = self.qkv[:, : H_q * d].unflatten(1, (H_q, d))
        self.k = self.qkv[:, H_q * d : (H_q + H_kv) * d].unflatten(1, (H_kv, d))
        self.v = self.qkv[:, (H_q + H_kv) * d : (H_q + 2 * H_kv) * d].unflatten(1, (H_kv, d))
        half = self.rot // 2
        self.axes = [0] * half if axes is None else axes
        n_axes = max(self.axes) + 1
        self.positions = torch.randint(-top, top, (n_axes, n), generator=g, device="cuda", dtype=torch.int32)
        self.inv_freq = (1e4 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)).float()
        self.rotary = pkv.Rotary(self.inv_freq, interleaved=interleaved, axes=self.axes)
        self.slots = torch.randperm(self.blocks * B, generator=g, device="cuda")[:n].to(torch.int32)
        shape = (self.blocks, L, H_kv, B, d)
        fill = torch.randint(0, 120, shape, generator=g, device="cuda")
        self.kp, self.vp = fill.to(STORE[dtype]), (fill + 1).to(STORE[dtype])
        self.q_out = torch.full((n, H_q, d), float("nan"), dtype=ACT[dtype], device="cuda")
        self.kp0, self.vp0 = self.kp.clone(), self.vp.clone()
        self.q0, self.k0, self.v0 = (x.double().cpu().numpy() for x in (self.q, self.k, self.v))
        self.slack = 2.0**-20 if top <= 1 << 20 else 2.0**-19

    def call(self, **kw):
        a = dict(q=self.q, k_new=self.k, v_new=self.v, positions=self.positions, slot_mapping=self.slots, q_out=self.q_out)
        a.update(kw)
        pkv.pkv_append_kv_rotary(self.pool, self.layer, self.rotary, a["q"], a["k_new"], a["v_new"], a["positions"],
                                 a["slot_mapping"], a["q_out"], self.kp, self.vp)

    def rotated(self, x):
        """(rotated x, radius of each element's pair), 64 bits."""
        half = self.rot // 2
        w = self.positions.cpu().numpy().astype(np.float64)[self.axes] * self.inv_freq.cpu().numpy().astype(np.float64)[:, None]
        c, s = np.cos(w).T[:, None], np.sin(w).T[:, None]  # [n, 1, half]
        i1 = np.arange(half) * 2 if self.interleaved else np.arange(half)
        i2 = i1 + 1 if self.interleaved else i1 + half
        y, r = x.copy(), np.zeros_like(x)
        y[..., i1], y[..., i2] = x[..., i1] * c - x[..., i2] * s, x[..., i2] * c + x[..., i1] * s
        r[..., i1] = r[..., i2] = np.hypot(x[..., i1], x[..., i2])
        return y, r

    def check_near(self, got, ref, radius, dtype):
        t = ACT[dtype]
        got = got.double().cpu().numpy()
        tol = radius * self.slack + np.abs(ref) * torch.finfo(t).eps / 2 + torch.finfo(t).tiny * torch.finfo(t).eps
        exact = radius == 0  # elements past rotary_dim pass as they are
        assert np.array_equal(got[exact], ref[exact])
        assert np.all(np.abs(got - ref) <= tol * (1 + 2.0**-7)), np.max(np.abs(got - ref) / tol)

    def rows_of(self, pool):
        """A pool's layer as one row per slot [slots][H_kv][d]."""
        return pool[:, self.layer].permute(0, 2, 1, 3).flatten(0, 1)

    def check(self, q=True, rows=None):
        pkv.pkv_check_device_error()
        if q:
            self.check_near(self.q_out, *self.rotated(self.q0), self.dtype if self.dtype != "e4m3" else "bf16")
        rows = slice(None) if rows is None else rows
        at = self.slots.long()[rows]
        y, r = (x[rows] for x in self.rotated(self.k0))
        kr, vr = self.rows_of(self.kp)[at], self.rows_of(self.vp)[at]
        if self.dtype == "e4m3":
            ref = np.clip(y / SCALES[0], -448, 448)
            got = kr.view(torch.float8_e4m3fn).double().cpu().numpy()
            tol = np.maximum(np.abs(ref) * 2.0**-4, 2.0**-10) * (1 + 2.0**-10) + r / SCALES[0] * self.slack
            assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) / tol)
            codes = (self.v[rows].float() / SCALES[1]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            assert torch.equal(vr, codes)
        else:
            self.check_near(kr, y, r, self.dtype)
            assert torch.equal(vr, self.v[rows])
        # every other slot and layer as it was
        for now, was in ((self.kp, self.kp0), (self.vp, self.vp0)):
            now, was = now.clone(), was.clone()
            for x in (now, was):
                x[:, self.layer].permute(0, 2, 1, 3)[at // self.B, at % self.B] = 0
            assert bool((now == was).all())


HALVES_3 = [0] * 8 + [1] * 12 + [2] * 12


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16", "e4m3"])
@pytest.mark.parametrize("kw", [
    dict(n=1),
    dict(n=37, H_q=64, H_kv=8, d=128),
    dict(n=300, H_q=7, H_kv=7, d=128, interleaved=True),
    dict(n=65, H_q=12, H_kv=4, d=96, rot=64, B=24),                      # part of the head rotated
    dict(n=19, H_q=3, H_kv=1, d=40, rot=6, interleaved=True, B=5),       # nothing a multiple of a vector
    dict(n=33, d=64, axes=HALVES_3),                                     # three axes
    dict(n=33, d=64, axes=[(2 * i) % 3 for i in range(32)], interleaved=True),
    dict(n=50, H_q=4, H_kv=2, d=256, B=32, L=2, layer=1),
    dict(n=21, d=64, top=2**31 - 1),                                     # any int32 position
    dict(n=21, d=64, pad=4),                                             # rows not on 16-byte boundaries
    dict(n=1100, H_q=2, H_kv=1, d=16),
], ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items() if k != "axes")[:40])
def test_against_the_definition(dtype, kw):
    c = Case(dtype, **kw)
    c.call()
    c.check()


@pytest.mark.parametrize("dtype", ["f16", "e4m3"])
def test_many_tokens(dtype):
    c = Case(dtype, n=4099, H_q=16, H_kv=4, d=128)
    c.call()
    c.check()


def test_in_place_keys_only_and_nothing():
    c = Case("bf16", n=40, H_q=16, H_kv=2, d=128)
    c.call(q_out=c.q)  # strided rows, rotated where they lie
    c.q_out = c.q
    c.check()
    assert torch.equal(c.v.double().cpu(), torch.from_numpy(c.v0))  # the row's other parts are untouched
    c = Case("bf16", n=40, H_q=16, H_kv=2, d=128)
    c.call(q=None, q_out=None)
    c.check(q=False)
    assert torch.isnan(c.q_out).all()
    c = Case("bf16", n=0)
    c.call()
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16", "e4m3"])
def test_position_zero_is_a_plain_append(dtype):
    c = Case(dtype, n=70, H_q=8, H_kv=4, d=128)
    c.positions.zero_()
    c.call()
    kp, vp = c.kp0.clone(), c.vp0.clone()
    pkv.pkv_append_kv(c.pool, 0, c.k.contiguous(), c.v.contiguous(), c.slots, kp, vp)
    as_values = (lambda x: x.view(torch.float8_e4m3fn).float()) if dtype == "e4m3" else (lambda x: x)
    assert torch.equal(as_values(c.kp), as_values(kp)) and torch.equal(c.vp, vp)
    assert torch.equal(c.q_out, c.q)


@pytest.mark.parametrize("pad", [0, 2])
def test_bad_slots_are_recorded_and_skipped(pad):
    c = Case("bf16", n=9, pad=pad)
    c.slots[2], c.slots[5] = -1, c.blocks * c.B
    c.call()
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_check_device_error()
    assert e.value.name == "PKV_ERR_DEVICE_CHECK" and "code 1" in str(e.value)
    c.check(rows=[0, 1, 3, 4, 6, 7, 8])  # the queries of all, the keys of the others


def test_offsets_past_32_bits():
    """A pool of more than 2^31 elements: slots at its far end."""
    H_kv, d, B = 8, 128, 16
    blocks = 2**31 // (H_kv * d * B) + 64
    pool = pkv.pkv_pool_create(1, H_kv, H_kv, d, B, "bf16", blocks)
    kp = torch.empty((blocks, 1, H_kv, B, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    n = 48
    k, v = (torch.randn((n, H_kv, d), device="cuda").to(torch.bfloat16) for _ in range(2))
    rotary = pkv.Rotary(torch.ones(d // 2, device="cuda"))
    slots = (blocks * B - 1 - 3 * torch.arange(n, device="cuda")).to(torch.int32)
    pkv.pkv_append_kv_rotary(pool, 0, rotary, None, k, v, torch.zeros(n, dtype=torch.int32, device="cuda"), slots, None, kp, vp)
    pkv.pkv_check_device_error()
    s = slots.long()
    assert torch.equal(kp[s // B, 0, :, s % B], k) and torch.equal(vp[s // B, 0, :, s % B], v)


def test_another_stream_and_a_replayed_graph():
    side = torch.cuda.Stream()
    c = Case("bf16", n=130, H_q=16, H_kv=2, d=128)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.call()
    side.synchronize()
    c.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call()
    for seed in (5, 6):
        d = Case("bf16", n=130, H_q=16, H_kv=2, d=128, seed=seed)
        for name in ("qkv", "positions", "slots", "kp", "vp"):
            getattr(c, name).copy_(getattr(d, name))
        c.kp0, c.vp0, c.q0, c.k0, c.v0 = d.kp0, d.vp0, d.q0, d.k0, d.v0
        graph.replay()
        c.check()


def test_refusals_of_the_binding():
    c = Case("bf16", n=12, H_q=8, H_kv=2, d=64)
    for kw, error, text in [
        (dict(q=c.q.float()), TypeError, "q is"),
        (dict(q=c.q.cpu()), TypeError, "CUDA"),
        (dict(q_out=None), TypeError, "q_out"),
        (dict(k_new=c.k[:, :1]), ValueError, "shape"),
        (dict(k_new=c.k.transpose(0, 1).contiguous().transpose(0, 1)), ValueError, "contiguous"),
        (dict(positions=c.positions.long()), TypeError, "positions"),
        (dict(positions=c.positions[:, :-1].contiguous()), ValueError, "positions"),
        (dict(slot_mapping=c.slots[:-1].contiguous()), ValueError, "positions"),
        (dict(slot_mapping=None), TypeError, "slot_mapping must"),
        (dict(positions=None), TypeError, "positions must"),
        (dict(k_new=None), TypeError, "k_new must"),
    ]:
        with pytest.raises(error, match=text):
            c.call(**kw)
    t = Case("bf16", n=12, d=64, axes=HALVES_3)
    for wrong in (t.positions.t().contiguous(), t.positions.reshape(-1)):  # as many positions, but in another order
        with pytest.raises(ValueError, match="positions"):
            t.call(positions=wrong)
    with pytest.raises(ValueError, match="entries"):
        pkv.Rotary(torch.ones(129, device="cuda"))
    with pytest.raises(ValueError, match="axes"):
        pkv.Rotary(torch.ones(8, device="cuda"), axes=[0, 1, 2, 4] * 2)
    with pytest.raises(TypeError):
        pkv.Rotary(torch.ones(8, device="cuda", dtype=torch.float64))
    with pytest.raises(pkv.PkvError, match="rotary_dim"):
        pkv.pkv_append_kv_rotary(c.pool, 0, pkv.Rotary(torch.ones(33, device="cuda")), c.q, c.k, c.v, c.positions, c.slots,
                                 c.q_out, c.kp, c.vp)
    with pytest.raises(ValueError, match="k_pool"):
        pkv.pkv_append_kv_rotary(c.pool, 0, c.rotary, c.q, c.k, c.v, c.positions, c.slots, c.q_out, c.kp[:-1], c.vp)
    assert torch.equal(c.kp, c.kp0) and torch.equal(c.vp, c.vp0) and torch.isnan(c.q_out).all()

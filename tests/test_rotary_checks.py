"""The C entry point of the rotary append refuses bad arguments before anything is launched (no GPU needed)."""
import ctypes

import pytest

import paged_kv_cache_80_gb300 as pkv

FAKE = 1 << 20  # an address that is never dereferenced: every call here fails on its arguments first


def call(pool, **kw):
    rot = pkv.RotaryConfig(FAKE, 64, 0, 1, (ctypes.c_uint8 * 128)())
    a = dict(layer=0, rotary=rot, q=FAKE, q_stride=512, k=FAKE, k_stride=128, v=FAKE, v_stride=128, positions=FAKE, slots=FAKE,
             n=3, q_out=FAKE, q_out_stride=512, kp=FAKE, vp=FAKE)
    for name in list(kw):
        if hasattr(rot, name):
            value = kw.pop(name)
            if name == "axis":
                rot.axis[5] = value
            else:
                setattr(rot, name, value)
    a.update(kw)
    L = pkv._L()
    rc = L.pkv_append_kv_rotary(pool.handle, a["layer"], ctypes.addressof(rot) if a["rotary"] is not None else None, a["q"],
                                a["q_stride"], a["k"], a["k_stride"], a["v"], a["v_stride"], a["positions"], a["slots"], a["n"],
                                a["q_out"], a["q_out_stride"], a["kp"], a["vp"], None)
    return L.pkv_status_name(rc).decode(), L.pkv_last_error_message().decode()


@pytest.mark.parametrize("kw,text", [
    (dict(rotary=None), "bad arguments"), (dict(n=-1), "bad arguments"),
    (dict(layer=-1), "layer"), (dict(layer=1), "layer"),
    (dict(rotary_dim=0), "rotary_dim"), (dict(rotary_dim=63), "rotary_dim"), (dict(rotary_dim=66), "rotary_dim"),
    (dict(interleaved=2), "interleaved"), (dict(n_axes=0), "n_axes"), (dict(n_axes=5), "n_axes"), (dict(axis=1), "axis"),
    (dict(inv_freq=None), "NULL"), (dict(k=None), "NULL"), (dict(v=None), "NULL"), (dict(positions=None), "NULL"),
    (dict(slots=None), "NULL"), (dict(kp=None), "NULL"), (dict(vp=None), "NULL"),
    (dict(q=None), "together"), (dict(q_out=None), "together"),
    (dict(k_stride=127), "stride"), (dict(v_stride=0), "stride"), (dict(q_stride=511), "stride"),
    (dict(q_out_stride=-512), "stride"), (dict(q_out_stride=520), "in place"),
    (dict(q=FAKE + 1), "aligned"), (dict(kp=FAKE + 1), "aligned"), (dict(positions=FAKE + 2), "aligned"),
], ids=lambda x: str(x)[:30])
def test_refused(kw, text):
    pool = pkv.pkv_pool_create(1, 8, 2, 64, 16, "bf16", 8)
    status, message = call(pool, **kw)
    assert status == "PKV_ERR_INVALID_ARG" and text in message


def test_no_tokens_is_no_work():
    pool = pkv.pkv_pool_create(1, 8, 2, 64, 16, "bf16", 8)
    assert call(pool, n=0, k=None, q=None)[0] == "PKV_OK"

"""Arguments that the rotating appends and the 8-bit calls refuse on the host: nothing of these
touches a device, so they run without a GPU."""
import ctypes

import pytest
import torch

from paged_kv_cache_299_gb300 import binding as pa

P = ctypes.c_void_p
FAKE = P(0x1000)  # never dereferenced
ODD = P(0x1008)


def desc(nb=4, hkv=8, d=64, bs=16):
    return pa.CacheDesc(nb, hkv, d, bs)


def append(q8, **kw):
    a = dict(q=FAKE, qs=2048, qo=FAKE, qos=2048, hq=32, k=FAKE, ks=512, v=FAKE, vs=512, cs=FAKE, npos=100,
             inter=0, bt=FAKE, mb=4, ctx=FAKE, qsl=FAKE, seqs=2, tokens=5, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE,
             cd=desc())
    a.update(kw)
    scales = (a["ksc"], a["vsc"]) if q8 else ()
    f = pa.load().pa_rope_append_q8 if q8 else pa.load().pa_rope_append
    return f(a["q"], a["qs"], a["qo"], a["qos"], a["hq"], a["k"], a["ks"], a["v"], a["vs"], a["cs"], a["npos"],
             a["inter"], a["bt"], a["mb"], a["ctx"], a["qsl"], a["seqs"], a["tokens"], a["kc"], a["vc"], *scales,
             a["cd"], None, None)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=None), dict(kc=None), dict(vc=None), dict(bt=None), dict(ctx=None), dict(q=None),
    dict(qo=None), dict(q=ODD), dict(qo=ODD), dict(k=ODD), dict(v=ODD), dict(cs=ODD), dict(kc=ODD), dict(vc=ODD),
    dict(qs=2044), dict(qs=2040), dict(ks=511), dict(ks=504), dict(vs=8), dict(qos=0), dict(hq=-1), dict(hq=4096),
    dict(npos=0), dict(tokens=-1), dict(seqs=0), dict(seqs=-2), dict(mb=0), dict(qsl=None),
    dict(qs=4096), dict(hq=0), dict(cd=desc(nb=0)), dict(cd=desc(hkv=65))])
def test_append_refuses(q8, bad):
    assert append(q8, **bad) == pa.PA_ERR_INVALID_ARG
    assert pa.load().pa_last_error() != b""


@pytest.mark.parametrize("q8", [False, True])
def test_append_unsupported_and_empty(q8):
    assert append(q8, cd=desc(d=128)) == pa.PA_ERR_UNSUPPORTED
    assert append(q8, cd=desc(bs=32)) == pa.PA_ERR_UNSUPPORTED
    assert append(q8, tokens=0, k=None, v=None, kc=None, vc=None, bt=None, ctx=None) == pa.PA_OK


def test_append_without_angles():
    assert append(False, cs=None) == pa.PA_ERR_INVALID_ARG
    assert append(True, cs=None) == pa.PA_ERR_INVALID_ARG  # query rows that nothing would rotate
    assert b"rotates" in pa.load().pa_last_error()
    for bad in (dict(ksc=None), dict(vsc=None), dict(ksc=P(0x1002)), dict(vsc=P(0x1001))):
        assert append(True, **bad) == pa.PA_ERR_INVALID_ARG


def decode(**kw):
    a = dict(out=FAKE, q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, cd=desc(), bt=FAKE, mb=4, ctx=FAKE, seqs=2, hq=32,
             scale=0.125, max_ctx=64, ws=FAKE, wb=1 << 30, flags=0)
    a.update(kw)
    return pa.load().pa_decode_q8(a["out"], a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["cd"], a["bt"], a["mb"],
                                  a["ctx"], a["seqs"], a["hq"], a["scale"], a["max_ctx"], a["ws"], a["wb"],
                                  a["flags"], None, None)


def test_decode_refuses():
    inv, uns = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED
    for name in ("out", "q", "kc", "vc", "ks", "vs", "bt", "ctx"):
        assert decode(**{name: None}) == inv, name
    for name in ("out", "q", "kc", "vc"):
        assert decode(**{name: ODD}) == inv, name
    assert decode(ks=P(0x1002)) == inv and decode(vs=P(0x1002)) == inv
    assert decode(hq=24) == uns and decode(hq=0) == inv and decode(hq=30) == inv
    assert decode(seqs=-1) == inv and decode(seqs=5000) == uns and decode(seqs=0) == pa.PA_OK
    assert decode(mb=0) == inv and decode(max_ctx=-1) == inv
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert decode(scale=s) == inv
    assert decode(flags=2) == inv and decode(flags=0x8000) == inv
    assert decode(cd=desc(d=32)) == uns and decode(cd=desc(bs=8)) == uns
    assert pa.pa_decode_q8_workspace_size(2, 8, 24, 64) == 0
    assert pa.pa_decode_q8_workspace_size(0, 8, 32, 64) == 0
    assert pa.pa_decode_q8_workspace_size(-1, 8, 32, 64) == 0


def chunk(**kw):
    a = dict(out=FAKE, q=FAKE, qsl=FAKE, tokens=16, mq=8, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, cd=desc(), bt=FAKE,
             mb=4, ctx=FAKE, seqs=2, hq=32, scale=0.125)
    a.update(kw)
    return pa.load().pa_prefill_chunk_q8(a["out"], a["q"], a["qsl"], a["tokens"], a["mq"], a["kc"], a["vc"], a["ks"],
                                         a["vs"], a["cd"], a["bt"], a["mb"], a["ctx"], a["seqs"], a["hq"],
                                         a["scale"], None, None)


def test_chunk_refuses():
    inv, uns = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED
    for name in ("out", "q", "qsl", "kc", "vc", "ks", "vs", "bt", "ctx"):
        assert chunk(**{name: None}) == inv, name
    for name in ("out", "q", "kc", "vc"):
        assert chunk(**{name: ODD}) == inv, name
    assert chunk(ks=P(0x1002)) == inv and chunk(vs=P(0x1003)) == inv
    assert chunk(hq=24) == uns and chunk(hq=9) == inv and chunk(mq=17) == inv and chunk(mq=-1) == inv
    assert chunk(seqs=-1) == inv and chunk(tokens=-1) == inv and chunk(mb=0) == inv
    assert chunk(seqs=0) == pa.PA_OK and chunk(tokens=0, mq=0) == pa.PA_OK
    assert chunk(scale=0.0) == inv and chunk(scale=float("nan")) == inv
    assert chunk(cd=desc(nb=1 << 24)) == uns  # 2^31 rows per pool
    assert chunk(cd=desc(d=128)) == uns
    assert chunk(seqs=1 << 26, tokens=1 << 20, mq=1 << 20) == uns  # work units past 2^31


def test_copy_refuses():
    f = pa.load().pa_copy_blocks_q8
    good = [FAKE, FAKE, FAKE, FAKE, desc(), FAKE, 3, None, None]
    for i in (0, 1, 2, 3, 5):
        bad = list(good)
        bad[i] = None
        assert f(*bad) == pa.PA_ERR_INVALID_ARG
    for i, p in ((0, ODD), (1, ODD), (2, P(0x1002)), (3, P(0x1001))):
        bad = list(good)
        bad[i] = p
        assert f(*bad) == pa.PA_ERR_INVALID_ARG
    bad = list(good)
    bad[6] = -1
    assert f(*bad) == pa.PA_ERR_INVALID_ARG
    assert f(None, None, None, None, desc(), None, 0, None, None) == pa.PA_OK
    assert f(FAKE, FAKE, FAKE, FAKE, desc(bs=8), FAKE, 3, None, None) == pa.PA_ERR_UNSUPPORTED


def test_status_of_values():
    assert pa.load().pa_status_string(pa.PA_ERR_DEVICE_VALUE) != b"unknown status"


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pa._need_rows(x, "key", 0)
    with pytest.raises(TypeError):
        pa._need_rows([1], "key", 0)
    codes = torch.zeros(2, 8, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        pa._need_q8(codes, codes, torch.ones(2, 8), torch.ones(2, 8), 0)


@pytest.mark.parametrize("stride", [1, 1001, 512, 4096, 20000])
def test_one_token_may_have_any_stride(stride):
    """The stride of a single token is never stepped over, and torch leaves it at anything; host
    tensors have device -1, so this much of the check runs without a GPU."""
    one = torch.empty(30000, dtype=torch.bfloat16).as_strided((1, 8, 64), (stride, 64, 1))
    assert pa._need_rows(one, "key", -1, 8) == 512
    two = torch.empty(30000, dtype=torch.bfloat16).as_strided((2, 8, 64), (stride, 64, 1))
    assert pa._need_rows(two, "key", -1, 8) == stride  # (the library refuses the bad ones)

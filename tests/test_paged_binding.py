"""What the paged cache's calls refuse, without a GPU: the C entry points with pointers that nothing reads, and the binding
against a library that records its calls."""
import ctypes

import numpy as np
import pytest
import torch

import alibi_positional_bias_gb300 as ab
from alibi_positional_bias_gb300 import _build

INVALID, UNSUPPORTED = ab.ALIBI_ERR_INVALID, ab.ALIBI_ERR_UNSUPPORTED
P, MIS, ODD = 0x10000, 0x10008, 0x10002


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ab.load()


def pages(**change):
    x = dict(k=P, v=P, k_page=2048, k_head=1024, k_slot=64, v_page=2048, v_head=1024, v_slot=64, table=P, pages=4, heads=2,
             slots=16, width=4, d=64)
    x.update(change)
    return ab.AlibiPages(*(x[n] for n, _ in ab.AlibiPages._fields_))


BAD_PAGES = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(table=None), INVALID), (dict(k=MIS), INVALID), (dict(v=MIS), INVALID),
    (dict(table=ODD), INVALID), (dict(pages=0), INVALID), (dict(heads=0), INVALID), (dict(slots=0), INVALID),
    (dict(width=0), INVALID), (dict(d=0), INVALID), (dict(pages=-1), INVALID), (dict(d=48), UNSUPPORTED),
    (dict(d=256), UNSUPPORTED), (dict(slots=4), UNSUPPORTED), (dict(slots=24), UNSUPPORTED), (dict(slots=2048), UNSUPPORTED),
    (dict(heads=385), UNSUPPORTED), (dict(width=(1 << 20) + 1), UNSUPPORTED), (dict(width=2 ** 31 - 1), UNSUPPORTED),
    (dict(k_slot=63), INVALID), (dict(k_slot=56), INVALID), (dict(v_head=68), INVALID), (dict(k_page=0), INVALID),
    (dict(v_page=-2048), INVALID), (dict(k_page=1 << 38), UNSUPPORTED)]


def append(lib, pg, k=(P, 64, 64, 64), v=(P, 64, 64, 64), pos=P, count=P, B=1, T=1, rot=None, q=None, q_out=None, H=0):
    rows = lambda r: None if r is None else ctypes.byref(ab.AlibiRows(*r))  # noqa: E731
    return lib.alibi_paged_append(rows(k), rows(v), pg, pos, count, B, T, rot, rows(q), q_out, H, None)


def decode(lib, pg, q=P, lens=P, out=P, lse=P, B=1, H=2, T=1, L=64, slopes=None):
    return lib.alibi_attn_decode_paged(q, pg, lens, out, lse, B, H, T, L, slopes, None)


@pytest.mark.parametrize("change,status", BAD_PAGES)
def test_caches_that_are_refused(lib, change, status):
    assert append(lib, pages(**change)) == status
    assert decode(lib, pages(**change)) == status


def test_no_cache(lib):
    assert append(lib, None) == INVALID and decode(lib, None) == INVALID


@pytest.mark.parametrize("change,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=(None, 64, 64, 64)), INVALID), (dict(k=(MIS, 64, 64, 64)), INVALID),
    (dict(v=(P, 64, 4, 64)), INVALID), (dict(k=(P, 64, -64, 64)), INVALID), (dict(pos=ODD), INVALID), (dict(count=ODD), INVALID),
    (dict(B=0), INVALID), (dict(T=0), INVALID), (dict(T=65), INVALID), (dict(T=-1), INVALID),
    (dict(q=(P, 64, 64, 64), q_out=P, H=2), INVALID),                                    # queries without a rotation
])
def test_appends_that_are_refused(lib, change, status):
    assert append(lib, pages(), **change) == status


def rotation(dims=64, interleaved=0, base=1e4, freqs=None):
    f = None if freqs is None else np.ascontiguousarray(freqs, dtype=np.float64)
    r = ab.AlibiRotation(dims, interleaved, base, None if f is None else f.ctypes.data_as(ctypes.POINTER(ctypes.c_double)))
    r.keep = f
    return r


@pytest.mark.parametrize("rot,change,status", [
    (rotation(dims=80), {}, INVALID), (rotation(dims=8), {}, INVALID), (rotation(dims=-16), {}, INVALID),
    (rotation(interleaved=2), {}, INVALID), (rotation(base=0.0), {}, INVALID), (rotation(base=float("nan")), {}, INVALID),
    (rotation(base=1e-9), {}, INVALID), (rotation(freqs=[np.inf] * 32), {}, INVALID), (rotation(freqs=[2e6] * 32), {}, INVALID),
    (rotation(), dict(q=(P, 64, 64, 64), q_out=None, H=2), INVALID), (rotation(), dict(q=(P, 64, 64, 64), q_out=MIS, H=2), INVALID),
    (rotation(), dict(q=(P, 64, 64, 64), q_out=P, H=0), INVALID), (rotation(), dict(q=(P, 60, 64, 64), q_out=P, H=2), INVALID),
    (rotation(), dict(q=(P, 64, 64, 64), q_out=P, H=385), UNSUPPORTED)])
def test_rotations_that_are_refused(lib, rot, change, status):
    assert append(lib, pages(), rot=ctypes.byref(rot), **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(q=MIS), INVALID), (dict(out=MIS), INVALID), (dict(lens=ODD), INVALID),
    (dict(lse=ODD), INVALID), (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(H=3), INVALID), (dict(T=0), INVALID),
    (dict(L=0), INVALID), (dict(L=65), INVALID), (dict(T=17), UNSUPPORTED), (dict(H=386), UNSUPPORTED),
    (dict(B=1 << 30, H=4), UNSUPPORTED)])
def test_decodes_that_are_refused(lib, change, status):
    assert decode(lib, pages(), **change) == status


def test_slopes_that_are_refused(lib):
    for bad in (-1.0, float("nan"), float("inf")):
        assert decode(lib, pages(), slopes=(ctypes.c_float * 2)(0.5, bad)) == INVALID


# ----------------------------------------------------------------- the binding

def test_tensors_that_are_refused():
    k = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    pools = (torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16),) * 2
    table = torch.zeros(1, 4, dtype=torch.int32)
    for call in (lambda: ab.alibi_paged_append(k, k, *pools, table), lambda: ab.alibi_attn_decode_paged(k, *pools, table)):
        with pytest.raises(ValueError):  # not CUDA tensors
            call()
    with pytest.raises(TypeError):
        ab.alibi_paged_append(None, k, *pools, table)
    with pytest.raises(TypeError):
        ab.alibi_attn_decode_paged([1], *pools, table)


class Tensor(torch.Tensor):
    """A CPU tensor that says it is on cuda:0."""
    is_cuda = True

    def get_device(self):
        return 0


def on(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Tensor)


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    f = Library()
    monkeypatch.setattr(ab, "_names", (torch.bfloat16, torch.uint8, torch.int32, torch.float32, lambda index: 0, lambda: 0, f))
    return f


def test_strides_are_passed_on(fake):
    pool = on(4, 16, 2, 64)
    kp = pool.transpose(1, 2)
    vp = on(4, 2, 16, 72)[..., 8:]
    k = on(1, 1, 2, 64).transpose(1, 2)
    ab.alibi_paged_append(k, k, kp, vp, on(1, 4, dtype=torch.int32))
    name, args = fake.calls[-1]
    pg = args[2]
    assert (pg.k_page, pg.k_head, pg.k_slot) == (2048, 64, 128)
    assert (pg.v_page, pg.v_head, pg.v_slot) == (2304, 1152, 72) and pg.v == vp.data_ptr()
    assert (pg.pages, pg.heads, pg.slots, pg.width, pg.d) == (4, 2, 16, 4, 64)
    assert (args[0].head, args[5:7]) == (64, (1, 1))
    # a dimension of one index has any stride
    one = on(4, 2, 16, 64).as_strided((4, 1, 16, 64), (1024, 3, 64, 1)).as_subclass(Tensor)
    ab.alibi_paged_append(on(1, 1, 1, 64), on(1, 1, 1, 64), one, one, on(1, 4, dtype=torch.int32))
    assert fake.calls[-1][1][2].k_head % 8 == 0 and fake.calls[-1][1][2].k_head >= 64


@pytest.mark.parametrize("L,ok", [(1, True), (64, True), (None, True), (0, False), (65, False), (2 ** 32 + 1, False), (-1, False)])
def test_the_bound(fake, L, ok):
    args = (on(1, 2, 64), on(4, 2, 16, 64), on(4, 2, 16, 64), on(1, 4, dtype=torch.int32))
    kw = dict(L=L, out=on(1, 2, 64), lse=on(1, 2, dtype=torch.float32))
    if ok:
        ab.alibi_attn_decode_paged(*args, **kw)
        assert fake.calls[-1][1][5:9] == (1, 2, 1, 64 if L is None else L)
    else:
        with pytest.raises(ab.AlibiError) as e:
            ab.alibi_attn_decode_paged(*args, **kw)
        assert e.value.status == INVALID and not fake.calls


def test_arguments_that_do_not_fit(fake):
    i32, f32 = torch.int32, torch.float32
    k, kp, table = on(2, 2, 3, 64), on(4, 2, 16, 64), on(2, 4, dtype=i32)
    q = on(2, 4, 1, 64)
    for error, call in [
        (ValueError, lambda: ab.alibi_paged_append(k, on(2, 2, 4, 64), kp, kp, table)),
        (TypeError, lambda: ab.alibi_paged_append(k, on(2, 2, 3, 64, dtype=f32), kp, kp, table)),
        (ValueError, lambda: ab.alibi_paged_append(k, k, kp, on(4, 2, 32, 64), table)),
        (ValueError, lambda: ab.alibi_paged_append(k, k, on(4, 3, 16, 64), on(4, 3, 16, 64), table)),
        (ValueError, lambda: ab.alibi_paged_append(k, k, on(4, 2, 16, 128), on(4, 2, 16, 128), table)),
        (ValueError, lambda: ab.alibi_paged_append(k, k, kp, kp, on(3, 4, dtype=i32))),
        (TypeError, lambda: ab.alibi_paged_append(k, k, kp, kp, on(2, 4, dtype=torch.int64))),
        (ValueError, lambda: ab.alibi_paged_append(k, k, kp, kp, on(2, 8, dtype=i32)[:, ::2])),
        (ValueError, lambda: ab.alibi_paged_append(k, k, kp, kp, table, pos=on(3, dtype=i32))),
        (TypeError, lambda: ab.alibi_paged_append(k, k, kp, kp, table, count=on(2, dtype=torch.int64))),
        (ValueError, lambda: ab.alibi_paged_append(on(2, 2, 3, 128)[..., ::2], k, kp, kp, table)),
        (ValueError, lambda: ab.alibi_paged_append(k, k, kp, kp, table, rotate=24)),
        (ValueError, lambda: ab.alibi_paged_append(k, k, kp, kp, table, rotate=80)),
        (ValueError, lambda: ab.alibi_paged_append(k, k, kp, kp, table, rotate=-16)),
        (ValueError, lambda: ab.alibi_paged_append(k, k, kp, kp, table, rotate=32, freqs=[1.0])),
        (ValueError, lambda: ab.alibi_paged_append(k, k, kp, kp, table, q=on(2, 4, 3, 64))),
        (ValueError, lambda: ab.alibi_paged_append(k, k, kp, kp, table, rotate=64, q=on(2, 4, 1, 64))),
        (ValueError, lambda: ab.alibi_paged_append(k, k, kp, kp, table, rotate=64, q_out=on(2, 4, 3, 64))),
        (ValueError, lambda: ab.alibi_attn_decode_paged(on(2, 4, 2, 64).transpose(1, 2), kp, kp, table)),
        (ValueError, lambda: ab.alibi_attn_decode_paged(q, kp, kp, table, out=on(2, 4, 2, 64))),
        (TypeError, lambda: ab.alibi_attn_decode_paged(q, kp, kp, table, out=q, lse=q)),
        (ValueError, lambda: ab.alibi_attn_decode_paged(q, kp, kp, table, out=q, lse=on(2, 4, 1, dtype=f32), lens=on(1, dtype=i32))),
        (ValueError, lambda: ab.alibi_attn_decode_paged(q, kp, kp, table, out=q, lse=on(2, 4, 1, dtype=f32), slopes=[1.0])),
        (ValueError, lambda: ab.alibi_attn_decode_paged(on(4, 64), kp, kp, table)),
    ]:
        with pytest.raises(error):
            call()
    assert not fake.calls


def prefill(lib, pg, q=P, lens=P, count=P, out=P, lse=P, B=1, H=2, T=1, L=64, slopes=None):
    return lib.alibi_attn_fwd_paged(q, pg, lens, count, out, lse, B, H, T, L, slopes, None)


@pytest.mark.parametrize("change,status", BAD_PAGES)
def test_caches_that_the_prefill_refuses(lib, change, status):
    assert prefill(lib, pages(**change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(q=MIS), INVALID), (dict(out=MIS), INVALID), (dict(lens=ODD), INVALID),
    (dict(count=ODD), INVALID), (dict(lse=ODD), INVALID), (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(H=3), INVALID),
    (dict(T=0), INVALID), (dict(L=0), INVALID), (dict(L=65), INVALID), (dict(T=(1 << 24) + 1), UNSUPPORTED), (dict(H=386), UNSUPPORTED),
    (dict(B=1 << 29, H=4), UNSUPPORTED), (dict(B=1 << 20, T=1 << 24), UNSUPPORTED),
    (dict(slopes=(ctypes.c_float * 2)(0.5, -1.0)), INVALID)])
def test_prefills_that_are_refused(lib, change, status):
    assert prefill(lib, pages(), **change) == status


def test_prefill_arguments_that_do_not_fit(fake):
    i32, f32 = torch.int32, torch.float32
    q, kp, table = on(2, 4, 3, 64), on(4, 2, 16, 64), on(2, 4, dtype=i32)
    lse = on(2, 4, 3, dtype=f32)
    for error, call in [
        (ValueError, lambda: ab.alibi_attn_fwd_paged(on(2, 4, 64), kp, kp, table)),
        (ValueError, lambda: ab.alibi_attn_fwd_paged(q.transpose(1, 2), kp, kp, table)),
        (ValueError, lambda: ab.alibi_attn_fwd_paged(q, kp, kp, table, out=q, lse=lse, count=on(3, dtype=i32))),
        (TypeError, lambda: ab.alibi_attn_fwd_paged(q, kp, kp, table, out=q, lse=lse, lens=on(2, dtype=f32))),
        (TypeError, lambda: ab.alibi_attn_fwd_paged(q, kp, kp, table, out=lse, lse=lse)),
        (ValueError, lambda: ab.alibi_attn_fwd_paged(q, kp, kp, table, out=q, lse=on(2, 4, dtype=f32))),
        (ab.AlibiError, lambda: ab.alibi_attn_fwd_paged(q, kp, kp, table, out=q, lse=lse, L=65)),
        (ab.AlibiError, lambda: ab.alibi_attn_fwd_paged(q, kp, kp, table, out=q, lse=lse, L=2 ** 32 + 5)),
    ]:
        with pytest.raises(error):
            call()
    assert not fake.calls
    ab.alibi_attn_fwd_paged(q, kp, kp, table, out=q, lse=lse)
    assert fake.calls[-1][1][6:10] == (2, 4, 3, 64)

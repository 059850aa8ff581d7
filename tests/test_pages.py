"""Refusals of the paged cache's entry points that the host makes before any
CUDA call, and the sizes they report (CPU)."""
import ctypes

import pytest

from shared_prefix_item_b200 import _lib as B

A = 1 << 20  # a pointer that no refused call follows


def pages(**over):
    f = dict(device=0, dtype=B.DTYPE_FP16, n_layers=2, n_kv_heads=2, head_dim=64, page_tokens=16, n_pages=32, n_seqs=8,
             max_pages=8, reserved=0, k=A, v=A, table=A, length=A, refs=A, status=A, workspace=A, workspace_bytes=1 << 20)
    f.update(over)
    return B.Pages(**f)


def batch(**over):
    f = dict(n=2, n_rows=4, max_rows=3, n_q_heads=4, causal=1, reserved=0, seq=A, offset=A, plan=A, plan_bytes=1 << 40)
    f.update(over)
    return B.PagesBatch(**f)


def resize(p, n=2, seq=A, length=A):
    return B.lib.duolm_pages_resize(ctypes.byref(p), n, seq, length, None)


def reason():
    return B.lib.duolm_last_error(None).decode()


@pytest.mark.parametrize("over, code", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(table=None), -1), (dict(length=None), -1), (dict(refs=None), -1),
    (dict(status=None), -1), (dict(workspace=None), -1), (dict(dtype=3), -1), (dict(dtype=-1), -1), (dict(n_layers=0), -1),
    (dict(n_kv_heads=0), -1), (dict(n_pages=0), -1), (dict(n_seqs=0), -1), (dict(max_pages=0), -1),
    (dict(page_tokens=4), -1), (dict(page_tokens=24), -1), (dict(page_tokens=512), -1), (dict(page_tokens=0), -1),
    (dict(head_dim=32), -1), (dict(head_dim=96), -1), (dict(head_dim=256), -1), (dict(head_dim=0), -1),
    (dict(dtype=B.DTYPE_FP32, head_dim=48), -1), (dict(dtype=B.DTYPE_FP32, head_dim=288), -1),
    (dict(n_seqs=(1 << 20) + 1), -5), (dict(max_pages=1 << 27), -5), (dict(n_pages=1 << 27), -5),
    (dict(k=A + 8), -1), (dict(v=A + 2), -1), (dict(status=A + 4), -1), (dict(workspace=A + 8), -1), (dict(table=A + 2), -1),
    (dict(length=A + 1), -1), (dict(refs=A + 2), -1), (dict(workspace_bytes=100), -5)])
def test_a_bad_cache_is_refused(over, code):
    p = pages(**over)
    assert resize(p) == code and reason()
    assert B.lib.duolm_pages_fork(ctypes.byref(p), 1, A, A, A, None) == code
    assert B.lib.duolm_pages_compact(ctypes.byref(p), A, A, A, None) == code
    assert B.lib.duolm_pages_check(ctypes.byref(p), None) == code
    b = batch()
    assert B.lib.duolm_pages_plan(ctypes.byref(p), ctypes.byref(b), None) == code
    assert B.lib.duolm_pages_plan_bytes(ctypes.byref(p), 1, 1, 1, 2) == code


def test_null_structures_and_arrays_are_refused():
    p, b = pages(), batch()
    r, rb = ctypes.byref(p), ctypes.byref(b)
    assert B.lib.duolm_pages_resize(None, 1, A, A, None) == -1
    assert resize(p, seq=None) == -1
    assert B.lib.duolm_pages_fork(r, 1, None, A, A, None) == -1
    assert B.lib.duolm_pages_fork(r, 1, A, None, A, None) == -1
    assert B.lib.duolm_pages_fork(r, 1, A, A, None, None) == -1
    assert B.lib.duolm_pages_compact(r, None, A, A, None) == -1
    assert B.lib.duolm_pages_compact(r, A, None, A, None) == -1
    assert B.lib.duolm_pages_compact(r, A, A, None, None) == -1
    assert B.lib.duolm_pages_plan(r, None, None) == -1
    assert B.lib.duolm_pages_attention(r, rb, 0, None, 256, 0.1, A, 256, None, None) == -1
    assert B.lib.duolm_pages_attention(r, rb, 0, A, 256, 0.1, None, 256, None, None) == -1


@pytest.mark.parametrize("n", [-1, 9])
def test_entry_counts_out_of_range_are_refused(n):
    p = pages()
    assert resize(p, n=n) == -1
    assert B.lib.duolm_pages_fork(ctypes.byref(p), n, A, A, A, None) == -1
    b = batch(n=n)
    assert B.lib.duolm_pages_plan(ctypes.byref(p), ctypes.byref(b), None) == -1


def test_nothing_to_do_is_no_error():
    p, b = pages(), batch(n=0, seq=None, offset=None, plan=None)
    r, rb = ctypes.byref(p), ctypes.byref(b)
    assert resize(p, n=0, seq=None) == 0
    assert B.lib.duolm_pages_fork(r, 0, None, None, None, None) == 0
    assert B.lib.duolm_pages_plan(r, rb, None) == 0
    assert B.lib.duolm_pages_write(r, rb, 0, None, 0, None, 0, None, 0, None, None, 0.0, None, 0, None, 0, None) == 0
    assert B.lib.duolm_pages_attention(r, rb, 1, None, 0, 0.1, None, 0, None, None) == 0


@pytest.mark.parametrize("over, code", [
    (dict(n_rows=-1), -1), (dict(max_rows=-1), -1), (dict(n_q_heads=0), -1), (dict(n_q_heads=3), -1),
    (dict(n_q_heads=130), -1), (dict(seq=None), -1), (dict(offset=None), -1), (dict(plan=None), -1),
    (dict(plan=A + 64), -1), (dict(n_rows=1 << 30), -5), (dict(n_rows=1 << 28), -5),
    (dict(n_rows=(1 << 30) + 1, n_q_heads=2), -5)])
def test_a_bad_batch_is_refused(over, code):
    p, b = pages(), batch(**over)
    r, rb = ctypes.byref(p), ctypes.byref(b)
    assert B.lib.duolm_pages_plan(r, rb, None) == code and reason()
    assert B.lib.duolm_pages_write(r, rb, 0, A, 256, A, 128, A, 128, None, None, 1e-6, None, 0, A, 256, None) == code
    assert B.lib.duolm_pages_attention(r, rb, 0, A, 256, 0.1, A, 256, None, None) == code


@pytest.mark.parametrize("over", [
    dict(layer=-1), dict(layer=2), dict(k=None), dict(v=None), dict(q_out=None), dict(q_stride=255), dict(k_stride=127),
    dict(v_stride=120), dict(q_out_stride=248), dict(q=A + 8), dict(k=A + 2), dict(v=A + 4), dict(q_out=A + 8),
    dict(q_stride=260), dict(k_stride=132), dict(rope=A + 8, rope_positions=4), dict(rope=A, rope_positions=0),
    dict(eps=-1.0), dict(eps=float("nan")), dict(q_gain=A + 4), dict(k_gain=A + 8)])
def test_bad_write_arguments_are_refused(over):
    f = dict(layer=0, q=A, q_stride=256, k=A, k_stride=128, v=A, v_stride=128, q_gain=None, k_gain=None, eps=1e-6,
             rope=None, rope_positions=0, q_out=A, q_out_stride=256)
    f.update(over)
    p, b = pages(), batch()
    assert B.lib.duolm_pages_write(ctypes.byref(p), ctypes.byref(b), *f.values(), None) == -1
    assert "pages_write" in reason()


@pytest.mark.parametrize("over", [
    dict(layer=-1), dict(layer=2), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(q_stride=248), dict(out_stride=248), dict(q=A + 8), dict(out=A + 2), dict(q_stride=260), dict(out_stride=257)])
def test_bad_attention_arguments_are_refused(over):
    f = dict(layer=0, q=A, q_stride=256, scale=0.125, out=A, out_stride=256, lse=None)
    f.update(over)
    p, b = pages(), batch()
    assert B.lib.duolm_pages_attention(ctypes.byref(p), ctypes.byref(b), *f.values(), None) == -1
    assert "pages_attention" in reason()


def test_workspace_bytes():
    assert B.PagedCache.workspace_bytes(32, 8) > 0
    assert B.PagedCache.workspace_bytes(1 << 16, 8) > B.PagedCache.workspace_bytes(32, 8)
    for bad in ((0, 1), (1, 0), (1 << 31, 1), (1, (1 << 20) + 1)):
        with pytest.raises(B.DuolmError):
            B.PagedCache.workspace_bytes(*bad)


def test_a_cache_of_host_arrays_is_refused():
    import torch
    k = torch.zeros(1, 4, 1, 16, 64, dtype=torch.float16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        B.PagedCache(k, k.clone(), torch.zeros(2, 2, dtype=torch.int32), i[:2], i, i, torch.zeros(1 << 12, dtype=torch.uint8))
    with pytest.raises(ValueError, match="alike"):
        B.PagedCache(k, k[:, :2], torch.zeros(2, 2, dtype=torch.int32), i[:2], i, i, torch.zeros(1 << 12, dtype=torch.uint8))

"""The compiled calls of the drafted trees let other Python threads run while the library works."""
import ctypes
import threading
import time

import pytest

from test_gpu_tree import BASE, i32, nb, setup  # noqa: F401 (nb is a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

NAMES = ("ne_attn_paged_plan_ex", "ne_attn_kv_append_slots", "ne_attn_decode_tree", "ne_attn_decode_tree_workspace_size",
         "ne_attn_kv_keep_paged")


def test_interpreter_lock_is_released(nb):
    """PyGILState_Check in the place of every entry point: as their status, 1 where the thread holds the lock, 0 where not."""
    s = setup([40, 20], [4, 4], 4, 4, 2, 64, 16, seed=1)
    k = s["q"][:, 0, :2].contiguous()
    held = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
    bind = nb._compiled()
    bind.init(dict({n: held for n in NAMES}, OutOfMemoryError=torch.OutOfMemoryError))
    try:
        nb.paged_plan(s["table"].clone(), i32([0]), i32([3, 2]), i32([0, 0]), i32([40, 20]), i32([0, 0]), 1, 16)
        nb.kv_append_slots(k, k, s["kp"], s["vp"], i32([-1, -1]), i32([0, 0]), 200)
        nb.attn_decode_tree(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["parents"])
        nb.kv_keep_paged(s["kp"], s["vp"], s["table"], s["lens"], 4, i32([[0], [1]]), i32([1, 1]))
    finally:
        real = {n: ctypes.cast(getattr(nb.lib(), n), ctypes.c_void_p).value for n in NAMES}
        bind.init(dict(real, OutOfMemoryError=torch.OutOfMemoryError))
    assert nb.attn_decode_tree(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["parents"])[1].isfinite().all()
    nb.check_status()


def test_a_waiting_call_holds_no_one_up(nb):
    """A thread clears a status and so waits for the device, with the library's mutex; a second one's call waits for that; the
    main thread goes on all the while."""
    k = torch.ones((2, 1, 32), device="cuda").bfloat16()
    kp, vp = nb.paged_cache(4, 16, 1, 32, "cuda")
    slots, pos, bad = i32([1, 2]), i32([0, 1]), i32([64, 1])
    append = lambda at: nb.kv_append_slots(k, k, kp, vp, at, pos, 10)
    append(slots)
    append(bad)
    torch.cuda.synchronize()
    times, results = {}, {}

    def clear():
        results["status"] = nb.status_of_last_kernels()

    def wait():
        t = time.perf_counter()
        append(slots)
        times["wait"] = time.perf_counter() - t
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        torch.cuda._sleep(1_600_000_000)  # 0.8 s at 2 GHz
    threads = [threading.Thread(target=clear), threading.Thread(target=wait)]
    threads[0].start()
    time.sleep(0.1)
    gap, last = 0.0, time.perf_counter()
    threads[1].start()  # may already wait for the interpreter
    while threads[1].is_alive():
        time.sleep(0.001)
        now = time.perf_counter()
        gap, last = max(gap, now - last), now
    for t in threads:
        t.join()
    assert results["status"] == -8 and times["wait"] > 0.3, times  # it did wait
    assert gap < 0.15
    nb.check_status()

"""The helper lets other Python threads run while it allocates (an allocation may wait for the GPU, and what the GPU waits
for may be theirs to enqueue)."""
import sys
import threading
import time

import torch


def test_other_threads_run_during_an_allocation():
    import fine_grained_blockwise_amd as fgb
    empties, t, specs = fgb._tensors.empties, torch.zeros(1), [(0, 4)] * 8
    ran, kept, go = [], [], threading.Event()  # (kept: freeing a tensor lets others run, too)

    def other():
        go.wait()
        ran.append(1)
    thread = threading.Thread(target=other)
    thread.start()
    time.sleep(0.2)  # (it waits)
    before = sys.getswitchinterval()
    sys.setswitchinterval(1000.0)  # from here on a thread runs only where another one lets it
    try:
        go.set()
        while not ran and len(kept) < 5000:
            kept.append(empties(t, *specs))
        seen = bool(ran)
    finally:
        sys.setswitchinterval(before)
    thread.join()
    assert seen

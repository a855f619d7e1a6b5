"""Calls through _marshal.so that need a device to get as far as the library."""
import ctypes
import subprocess
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

# Stands in for the library's function: tells that it has begun, then waits (2 s
# at most) for another thread to answer.  Fails (3) if none could.
WAITS = """
#include <time.h>
volatile int begun, answered;
int waits(void)
{
    begun = 1;
    for (int i = 0; i < 2000 && !answered; ++i) {
        struct timespec t = {0, 1000000};
        nanosleep(&t, 0);
    }
    return answered ? 0 : 3;
}
"""


def _rope_tensors(tokens=2):
    h = dict(dtype=torch.float16, device="cuda")
    long = torch.zeros(tokens, dtype=torch.int64, device="cuda")
    return [torch.zeros(tokens, 8, 128, **h), torch.zeros(tokens, 8, 128, **h),
            torch.zeros(tokens, 2, 128, **h), torch.zeros(tokens, 2, 128, **h),
            torch.zeros(3, 16, 2, 128, **h), torch.zeros(3, 16, 2, 128, **h), long, long.clone(),
            torch.zeros(4, 128, device="cuda")]


def test_other_threads_run_during_a_call(tmp_path):
    from paged_kv_cache_415_b200 import binding as B
    (tmp_path / "waits.c").write_text(WAITS)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-o", str(tmp_path / "waits.so"),
                    str(tmp_path / "waits.c")], check=True)
    lib = ctypes.CDLL(str(tmp_path / "waits.so"))
    begun, answered = (ctypes.c_int.in_dll(lib, n) for n in ("begun", "answered"))

    def answer():
        while not begun.value:
            pass
        answered.value = 1

    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value
    names = ("rope_append", "latent_append", "latent_decode", "latent_prefill")
    tensors = _rope_tensors()
    assert B._marshal.rope_append
    from paged_kv_cache_415_b200 import _marshal as module
    module.bind(*[address(lib.waits)] * 4)
    try:
        other = threading.Thread(target=answer)
        other.start()
        B.pa_rope_append(*tensors)                   # raises if nobody answered
        other.join()
    finally:
        begun.value = 1
        module.bind(*(address(getattr(B.LIB, "pa_" + n)) for n in names))
    B.pa_rope_append(*tensors)
    torch.cuda.synchronize()

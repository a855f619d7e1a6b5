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


def test_strides_of_single_rows_do_not_matter():
    """One token, and one head: torch gives the axis of one element whatever
    stride a view came by, and it is not used."""
    from paged_kv_cache_415_b200 import binding as B
    odd = lambda t, axes: torch.as_strided(t, t.shape, [3 if i in axes else s
                                                        for i, s in enumerate(t.stride())])
    args = _rope_tensors(1)
    for i in range(4):
        args[i].normal_()
    args[8].copy_(torch.rand_like(args[8]))
    want = [a.clone() for a in args]
    B.pa_rope_append(*want)
    got = [odd(a, (0,)) if i < 4 else a for i, a in enumerate(args)]
    B.pa_rope_append(*got)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and got[0].any()
    h = dict(dtype=torch.bfloat16, device="cuda")
    q, rows = torch.randn(1, 1, 64, **h), torch.randn(1, 576, **h)
    long, table = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.rand(4, 64, device="cuda")
    outs, pools = [torch.zeros_like(q) for _ in range(2)], [torch.zeros(2, 16, 576, **h) for _ in range(2)]
    B.pa_latent_append(outs[0], q, rows, pools[0], long, long, table)
    B.pa_latent_append(odd(outs[1], (0, 1)), odd(q, (0, 1)), odd(rows, (0,)), pools[1], long, long,
                       table)
    assert torch.equal(*outs) and torch.equal(*pools) and outs[0].any()
    with pytest.raises(B.PAError):                   # of two tokens it does
        B.pa_latent_append(None, None, torch.as_strided(torch.zeros(1200, **h), (2, 576), (580, 1)),
                           pools[0], long.repeat(2), long.repeat(2), table)

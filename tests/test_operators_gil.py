"""The operators' calls let other Python threads run while the library's entry
point does: one that waits (for room in a stream's queue, for a callback that
needs the interpreter) holds nobody up."""
import ctypes
import shutil
import subprocess
import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

# stands in for each entry point: answers 0 once another thread has set the
# flag, 77 if that takes more than two seconds
SOURCE = r"""
#include <unistd.h>
volatile int flag;
static int wait_for_flag(void)
{
    for (int i = 0; i < 2000; ++i) {
        if (flag)
            return 0;
        usleep(1000);
    }
    return 77;
}
int two(const void* a, void* s) { (void)a, (void)s; return wait_for_flag(); }
int four(void* c, const void* b, const void* a, void* s) { (void)c, (void)b, (void)a, (void)s; return wait_for_flag(); }
"""


@pytest.fixture(scope="module")
def waiting(tmp_path_factory):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc is not installed")
    at = tmp_path_factory.mktemp("waiting")
    (at / "waiting.c").write_text(SOURCE)
    subprocess.run([gcc, "-std=gnu99", "-O1", "-shared", "-fPIC", str(at / "waiting.c"), "-o",
                    str(at / "waiting.so")], check=True)
    return ctypes.CDLL(str(at / "waiting.so"))


@pytest.mark.parametrize("which", ("rmsnorm", "reduce_scatter_rmsnorm", "rmsnorm_backward"))
def test_other_threads_run_during_a_call(waiting, which):
    from collective_communication_ring_amd import api
    dev = torch.device("cuda:0")
    x, w, y = torch.ones((2, 8), device=dev), torch.ones(8, device=dev), torch.ones((2, 8), device=dev)
    rstd, dw = torch.ones(2, device=dev), torch.ones((1, 8), device=dev)
    comm = api.Comm(2, 16, "float32", device=dev)
    send, y2 = torch.ones((2, 16), device=dev), torch.ones((2, 8), device=dev)
    ws = api.rmsnorm_backward_workspace(1, 2, 8, dev)
    torch.cuda.synchronize()
    call = {"rmsnorm": lambda: api.rmsnorm(x, w, y),
            "reduce_scatter_rmsnorm": lambda: comm.reduce_scatter_rmsnorm(send, w, y2),
            "rmsnorm_backward": lambda: api.rmsnorm_backward(x, x, w, rstd, y, dw, workspace=ws)}[which]
    call()  # the library's own
    flag = ctypes.c_int.in_dll(waiting, "flag")
    flag.value = 0
    two, four = (ctypes.cast(f, ctypes.c_void_p).value for f in (waiting.two, waiting.four))
    binding = api.binding()

    def set_flag():
        time.sleep(0.05)
        flag.value = 1
    other = threading.Thread(target=set_flag)
    try:
        binding.init(two, four, two)
        other.start()
        call()  # 77 would raise ArError
    finally:
        api._bound = None
        api.binding()
        other.join()
    call()
    torch.cuda.synchronize()
    comm.close()

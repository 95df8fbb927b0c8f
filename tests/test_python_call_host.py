"""What the C++ binding puts around each call, in a module of its own: other
threads run meanwhile, exceptions come back as a status, and a thread that ends
while Python shuts down does not take the process with it."""
import os
import subprocess
import sys
import sysconfig

import pytest

mod = pytest.importorskip("expert_grouping_dispatch_amd")
CSRC = os.path.join(os.path.dirname(mod.LIB_PATH), "csrc")
SOURCE = """
#include "python_call.h"
#include <stdexcept>
#include <unistd.h>
static PyObject* rest(PyObject*, PyObject* const*, Py_ssize_t) {
  return moe::unlocked([] { return usleep(20000) == 0 ? 7 : 8; });
}
static PyObject* fail(PyObject*, PyObject* const*, Py_ssize_t n) {
  if (n == 0) throw std::runtime_error("no");
  PyErr_SetString(PyExc_ValueError, "no");
  throw 1;
}
#define M(f) {#f, reinterpret_cast<PyCFunction>(&moe::guarded<f>), METH_FASTCALL, nullptr}
static PyMethodDef methods[] = {M(rest), M(fail), {nullptr, nullptr, 0, nullptr}};
static PyModuleDef module = {PyModuleDef_HEAD_INIT, "calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};
PyMODINIT_FUNC PyInit_calls() { return PyModule_Create(&module); }
"""


@pytest.fixture(scope="module")
def at(tmp_path_factory):
    d = tmp_path_factory.mktemp("calls")
    (d / "calls.cpp").write_text(SOURCE)
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", CSRC, "-I", sysconfig.get_paths()["include"],
                        str(d / "calls.cpp"), "-o", str(d / "calls.so")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return d


def _run(at, code):
    r = subprocess.run([sys.executable, "-c", code], cwd=at, capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, (r.returncode, r.stderr)
    return r.stdout


def test_status_and_exceptions(at):
    assert _run(at, "import calls; print(calls.rest(), calls.fail(), calls.fail(1), calls.rest())") == "7 -1 -1 7\n"


def test_other_threads_run_meanwhile(at):
    assert _run(at, """
import calls, sys, threading
turns = []
sys.setswitchinterval(1000)
thread = threading.Thread(target=lambda: turns.append(1), daemon=True)
thread._started.set()  # start() would wait for the thread, and so let it run
threading._start_new_thread(thread._target, ())
before = len(turns)
calls.rest()
print(before, len(turns))
""") == "0 1\n"


def test_a_thread_that_is_in_a_call_when_python_ends(at):
    _run(at, """
import calls, sys, threading, time
class Slow:  # goes while Python shuts down, and lets other threads ask for the lock
    def __del__(self, sleep=time.sleep):
        sleep(0.1)
sys.slow = Slow()
def loop():
    while True:
        calls.rest()
threading.Thread(target=loop, daemon=True).start()
time.sleep(0.03)
""")

"""Calls of the library's operators with the runtime's launches replaced (hip_stub.c): which kernels
a call launches, and what it answers when one of the runtime's calls fails.  No GPU is needed
and no address is dereferenced."""
import json
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))


def build(folder) -> str:
    lib = os.path.join(str(folder), "hip_stub.so")
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-o", lib, os.path.join(HERE, "hip_stub.c")],
                   check=True)
    return lib


def run(lib, calls):
    """calls: [name, keyword arguments, settings of stub_reset]; answers, in order, a dict of each
    call's status, its launches (name, grid x and y, threads, LDS bytes), the attributes it set
    and the error it leaves; then the names of all kernels."""
    p = subprocess.run([sys.executable, os.path.abspath(__file__), lib], input=json.dumps(calls),
                       capture_output=True, text=True, timeout=100)
    assert p.returncode == 0, p.stderr
    return json.loads(p.stdout)


def _main(lib):
    import ctypes
    stub = ctypes.CDLL(lib, mode=ctypes.RTLD_GLOBAL)  # before the runtime itself
    sys.path.insert(0, os.path.dirname(HERE))
    import expert_cache_offload_amd as m
    for f in (stub.stub_kernel, stub.stub_launch, stub.stub_attribute):
        f.restype = ctypes.c_char_p
    shape, value = (ctypes.c_uint * 5)(), ctypes.c_int()
    out = []
    for name, args, setting in json.load(sys.stdin):
        stub.stub_reset(setting.get("launch", 0), setting.get("attribute", 0),
                        setting.get("error", 0), setting.get("device", 0))
        status = m.MOE_OK
        try:
            getattr(m, name)(**args)
        except m.MoeError as e:
            status = e.status
        launches = []
        for i in range(stub.stub_launches()):
            kernel = stub.stub_launch(i, shape).decode()
            launches.append([kernel, shape[0], shape[1], shape[3], shape[4]])
        attributes = [[stub.stub_attribute(i, ctypes.byref(value)).decode(), value.value]
                      for i in range(stub.stub_attributes())]
        out.append(dict(status=status, launches=launches, attributes=attributes,
                        error=stub.stub_pending()))
    kernels = [stub.stub_kernel(i).decode() for i in range(stub.stub_kernels())]
    json.dump([out, kernels], sys.stdout)


if __name__ == "__main__":
    _main(sys.argv[1])

// latent_host.cpp -- the usual calls of latent.py without the interpreter in between.
//
// A Python extension module: each function takes the tensors of one call, checks that they are
// what the kernels take (bf16, on the current GPU, the layouts of include/kda.h), allocates the
// results and calls the library. Anything else, right or wrong (another device or stream,
// results of the caller's, a shape that does not fit), is answered with None: latent.py then
// goes through its own checks, which say what is wrong. In Python the same steps take the host
// 17 us for a decode and for a forward and 7.5 for a cache write, more than the 14, 7 and 3 that a
// token over a short cache, a few short prompts and a few tokens take the GPU; here 7.5, 5.8 and 2.6.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/kda.h"

namespace {

// the library's entry points, given by latent.py
struct Lib {
  decltype(&kda_latent_attn_fwd) fwd;
  decltype(&kda_latent_attn_bwd) bwd;
  decltype(&kda_latent_attn_bwd_workspace_size) bwd_ws;
  decltype(&kda_latent_cache_write) write;
  decltype(&kda_latent_cache_read) read;
  decltype(&kda_latent_decode) decode;
  decltype(&kda_latent_decode_workspace_size) decode_ws;
} lib;

constexpr int64_t DN = 128, DP = 64, DV = 128, DC = 512, DX = 576;

struct Unusual {};  // thrown: leave the call to latent.py

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_CheckExact(o)) throw Unusual{};
  return THPVariable_Unpack(o);
}

void need(bool ok) {
  if (!ok) throw Unusual{};
}

struct Here {  // the current device, where every tensor of a usual call is
  int index = c10::cuda::current_device();
  const at::Tensor& take(PyObject* o, at::ScalarType type) const {
    const at::Tensor& t = tensor(o);
    need(t.is_cuda() && t.get_device() == index && t.scalar_type() == type && t.layout() == at::kStrided);
    return t;
  }
  const at::Tensor& whole(PyObject* o, at::ScalarType type) const {
    const at::Tensor& t = take(o, type);
    need(t.is_contiguous());
    return t;
  }
  kda_stream_t stream() const {
    return reinterpret_cast<kda_stream_t>(c10::cuda::getCurrentCUDAStream(index).stream());
  }
};

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Unusual{};
  return v;
}

float scale_of(PyObject* o) {
  if (o == Py_None) return 0.f;
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Unusual{};
  const float f = static_cast<float>(v);
  if (!(f > 0.f && f <= 3.4028235e38f)) throw Unusual{};  // (0 would select the default)
  return f;
}

void* ptr(const at::Tensor& t) { return t.data_ptr(); }

PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }

template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

// packed or single inputs of the expanded form: [T, H, d] with more than one token and head
struct Expanded {
  const at::Tensor &q, &kn, &kp, &v;
  const int32_t *cu_q = nullptr, *cu_k = nullptr;
  kda_latent_shape s{};

  Expanded(const Here& here, PyObject* const* a)  // q, k_nope, k_pe, v, cu_q, cu_k, max_q, max_k, causal, scale
      : q(here.take(a[0], at::kBFloat16)), kn(here.take(a[1], at::kBFloat16)),
        kp(here.take(a[2], at::kBFloat16)), v(here.take(a[3], at::kBFloat16)) {
    need(q.dim() == 3 && kn.dim() == 3 && kp.dim() == 2 && v.dim() == 3);
    const int64_t T = q.size(0), Tk = kn.size(0), H = q.size(1);
    need(T > 1 && Tk > 1 && H > 1 && H <= 65535 && kn.size(1) == H && v.size(1) == H && v.size(0) == Tk &&
         kp.size(0) == Tk && q.size(2) == DN + DP && kn.size(2) == DN && kp.size(1) == DP && v.size(2) == DV);
    need(q.stride(2) == 1 && kn.stride(2) == 1 && kp.stride(1) == 1 && v.stride(2) == 1);
    need((a[4] == Py_None) == (a[5] == Py_None));
    if (a[4] != Py_None) {
      const at::Tensor &x = here.whole(a[4], at::kInt), &y = here.whole(a[5], at::kInt);
      need(x.dim() == 1 && y.dim() == 1 && x.numel() >= 2 && x.numel() == y.numel() && x.numel() <= 65536);
      cu_q = static_cast<const int32_t*>(ptr(x));
      cu_k = static_cast<const int32_t*>(ptr(y));
      s.n_seqs = static_cast<int32_t>(x.numel() - 1);
    }
    s.B = 1;
    s.H = static_cast<int32_t>(H);
    s.Tq = T;
    s.Tk = Tk;
    s.max_q = integer(a[6]);
    s.max_k = integer(a[7]);
    s.d_nope = DN;
    s.d_pe = DP;
    s.d_v = DV;
    s.q_token = q.stride(0);
    s.q_head = q.stride(1);
    s.k_token = kn.stride(0);
    s.k_head = kn.stride(1);
    s.pe_token = kp.stride(0);
    s.v_token = v.stride(0);
    s.v_head = v.stride(1);
    const int causal = PyObject_IsTrue(a[8]);
    need(causal >= 0);
    s.causal = causal;
    s.dtype = KDA_BF16;
    s.scale = scale_of(a[9]);
  }
};

PyObject* attn_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 10);
    const Here here;
    const Expanded x(here, a);
    at::Tensor out = at::empty({x.s.Tq, x.s.H, DV}, x.q.options());
    at::Tensor lse = at::empty({x.s.Tq, x.s.H}, x.q.options().dtype(at::kFloat));
    need(lib.fwd(ptr(x.q), ptr(x.kn), ptr(x.kp), ptr(x.v), x.cu_q, x.cu_k, ptr(out),
                 static_cast<float*>(ptr(lse)), &x.s, nullptr, here.stream()) == KDA_OK);
    return Py_BuildValue("(NN)", wrap(std::move(out)), wrap(std::move(lse)));
  });
}

PyObject* attn_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {  // the ten of attn_fwd, out, lse, d_out
  return guarded([&]() -> PyObject* {
    need(n == 13);
    const Here here;
    const Expanded x(here, a);
    const at::Tensor &out = here.whole(a[10], at::kBFloat16), &lse = here.whole(a[11], at::kFloat),
                     &g = here.whole(a[12], at::kBFloat16);
    const int64_t T = x.s.Tq, Tk = x.s.Tk, H = x.s.H;
    need(out.sizes() == at::IntArrayRef({T, H, DV}) && g.sizes() == out.sizes() &&
         lse.sizes() == at::IntArrayRef({T, H}));
    const size_t bytes = lib.bwd_ws(&x.s);
    need(bytes > 0);
    const auto o = x.q.options();
    at::Tensor dq = at::empty({T, H, DN + DP}, o), dkn = at::empty({Tk, H, DN}, o),
               dkp = at::empty({Tk, DP}, o), dv = at::empty({Tk, H, DV}, o);
    at::Tensor ws = at::empty({static_cast<int64_t>(bytes)}, o.dtype(at::kByte));
    need(lib.bwd(ptr(x.q), ptr(x.kn), ptr(x.kp), ptr(x.v), ptr(out), static_cast<float*>(ptr(lse)),
                 ptr(g), x.cu_q, x.cu_k, ptr(dq), ptr(dkn), ptr(dkp), ptr(dv), &x.s, ptr(ws), bytes,
                 nullptr, here.stream()) == KDA_OK);
    return Py_BuildValue("(NNNN)", wrap(std::move(dq)), wrap(std::move(dkn)), wrap(std::move(dkp)),
                         wrap(std::move(dv)));
  });
}

kda_latent_cache cache_of(const at::Tensor& t) {
  need(t.dim() == 3 && t.is_contiguous());
  const bool f8 = t.scalar_type() == at::kByte;
  need(t.size(2) == (f8 ? KDA_CACHE_E4M3_ROW_BYTES : DX) && t.size(1) <= 128);
  return kda_latent_cache{t.size(0), static_cast<int32_t>(t.size(1)), DC, DP,
                          f8 ? KDA_CACHE_E4M3 : KDA_CACHE_BF16};
}
const at::Tensor& cache(const Here& here, PyObject* o) {
  return here.take(o, tensor(o).scalar_type() == at::kByte ? at::kByte : at::kBFloat16);
}

PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {  // latent, k_pe, cache, slots
  return guarded([&]() -> PyObject* {
    need(n == 4);
    const Here here;
    const at::Tensor &c = here.take(a[0], at::kBFloat16), &pe = here.take(a[1], at::kBFloat16),
                     &t = cache(here, a[2]), &slots = here.whole(a[3], at::kLong);
    const kda_latent_cache cs = cache_of(t);
    need(c.dim() == 2 && pe.dim() == 2 && slots.dim() == 1);
    const int64_t T = c.size(0);
    need(T > 1 && pe.size(0) == T && slots.size(0) == T && c.size(1) == DC && pe.size(1) == DP &&
         c.stride(1) == 1 && pe.stride(1) == 1);
    need(lib.write(ptr(c), c.stride(0), ptr(pe), pe.stride(0), static_cast<int64_t*>(ptr(slots)), T,
                   ptr(t), &cs, nullptr, here.stream()) == KDA_OK);
    Py_RETURN_TRUE;
  });
}

PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {  // cache, block_table, cu_seqlens, total
  return guarded([&]() -> PyObject* {
    need(n == 4);
    const Here here;
    const at::Tensor &t = cache(here, a[0]), &table = here.whole(a[1], at::kInt), &cu = here.whole(a[2], at::kInt);
    const kda_latent_cache cs = cache_of(t);
    const int64_t total = integer(a[3]);
    need(table.dim() == 2 && cu.dim() == 1 && cu.numel() == table.size(0) + 1 && table.size(0) >= 1 &&
         table.size(0) < (1LL << 31) && total >= 0);
    at::Tensor out = at::empty({total, DX}, t.options().dtype(at::kBFloat16));
    need(lib.read(ptr(t), static_cast<int32_t*>(ptr(table)), table.size(1), static_cast<int32_t*>(ptr(cu)),
                  nullptr, static_cast<int32_t>(table.size(0)), total, ptr(out), &cs, nullptr,
                  here.stream()) == KDA_OK);
    return wrap(std::move(out));
  });
}

PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {  // q, cache, block_table, seq_lens, draft_mask, scale
  return guarded([&]() -> PyObject* {
    need(n == 6);
    const Here here;
    const at::Tensor &q = here.whole(a[0], at::kBFloat16), &t = cache(here, a[1]),
                     &table = here.whole(a[2], at::kInt), &lens = here.whole(a[3], at::kInt);
    const kda_latent_cache cs = cache_of(t);
    const int64_t d = q.dim();
    need((d == 3 || d == 4) && q.size(-1) == DX);
    const int64_t N = q.size(0), L = d == 4 ? q.size(1) : 1, H = q.size(-2);
    need(N <= 65535 && L <= 64 && H <= 1024 && table.dim() == 2 && table.size(0) == N && lens.dim() == 1 &&
         lens.size(0) == N);
    const int64_t* mask = nullptr;
    if (a[4] != Py_None) {
      const at::Tensor& m = here.whole(a[4], at::kLong);
      need(m.dim() == 2 && m.size(0) == N && m.size(1) == L);
      mask = static_cast<int64_t*>(ptr(m));
    }
    const kda_latent_decode_shape s{static_cast<int32_t>(N), static_cast<int32_t>(L), static_cast<int32_t>(H),
                                    table.size(1), KDA_BF16, scale_of(a[5])};
    const size_t bytes = lib.decode_ws(&s, &cs);
    need(bytes > 0);
    at::Tensor out = d == 4 ? at::empty({N, L, H, DC}, q.options()) : at::empty({N, H, DC}, q.options());
    at::Tensor ws = at::empty({static_cast<int64_t>(bytes)}, q.options().dtype(at::kByte));
    need(lib.decode(ptr(q), ptr(t), static_cast<int32_t*>(ptr(table)), static_cast<int32_t*>(ptr(lens)), mask,
                    ptr(out), nullptr, &s, &cs, ptr(ws), bytes, nullptr, here.stream()) == KDA_OK);
    return wrap(std::move(out));
  });
}

PyObject* bind(PyObject*, PyObject* args) {  // addresses: fwd, bwd, bwd_ws, write, read, decode, decode_ws
  unsigned long long p[7];
  if (!PyArg_ParseTuple(args, "KKKKKKK", p, p + 1, p + 2, p + 3, p + 4, p + 5, p + 6)) return nullptr;
  lib.fwd = reinterpret_cast<decltype(lib.fwd)>(p[0]);
  lib.bwd = reinterpret_cast<decltype(lib.bwd)>(p[1]);
  lib.bwd_ws = reinterpret_cast<decltype(lib.bwd_ws)>(p[2]);
  lib.write = reinterpret_cast<decltype(lib.write)>(p[3]);
  lib.read = reinterpret_cast<decltype(lib.read)>(p[4]);
  lib.decode = reinterpret_cast<decltype(lib.decode)>(p[5]);
  lib.decode_ws = reinterpret_cast<decltype(lib.decode_ws)>(p[6]);
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"attn_fwd", FAST(attn_fwd)},       {"attn_bwd", FAST(attn_bwd)},
                         {"cache_write", FAST(cache_write)}, {"cache_read", FAST(cache_read)},
                         {"decode", FAST(decode)},           {"bind", bind, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_latent_host", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__latent_host() { return PyModule_Create(&module); }

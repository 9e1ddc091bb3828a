// fa_binding.cpp -- the paged cache's calls for torch tensors, as a CPython
// extension module.  A decode step makes four calls whose kernels run for a few
// microseconds each; checking their three dozen tensors in Python and converting
// the arguments one by one took longer than that.  Here a call takes the tensors
// as they are, checks type, device, shape and layout, and calls the C interface
// (include/fa.h) on the stream given, or on torch's current one.  Returns the C
// call's status; what the C interface cannot see (a wrong dtype, shape or device)
// is a ValueError.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <exception>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "../../include/fa.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct BadTensor : std::invalid_argument {
    using std::invalid_argument::invalid_argument;
};

const Tensor &tensor_of(PyObject *obj, const char *name) {
    if (!THPVariable_Check(obj)) throw BadTensor(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(obj);
}

const Tensor *tensor_or_none(PyObject *obj, const char *name) { return obj == Py_None ? nullptr : &tensor_of(obj, name); }

// t is on `device`, of type `type` (or `other`) and of `shape` (-1: any size), and
// contiguous, or, with `strided`, contiguous in all but its first dimension.
void check(const char *name, const Tensor &t, c10::Device device, ScalarType type, std::initializer_list<int64_t> shape,
           bool strided = false, ScalarType other = ScalarType::Undefined) {
    bool fits = t.scalar_type() == type || t.scalar_type() == other;
    fits = fits && t.device() == device && t.dim() == (int64_t)shape.size();
    int64_t d = 0;
    if (fits)
        for (const int64_t n : shape) fits = fits && (n < 0 || t.size(d) == n), ++d;
    if (fits && !t.is_contiguous()) {
        fits = strided;
        int64_t step = 1;
        for (d = t.dim() - 1; fits && d > 0; --d) {
            fits = t.size(d) <= 1 || t.stride(d) == step;
            step *= t.size(d);
        }
    }
    if (fits) return;
    std::string want = std::string(name) + " must be a " + c10::toString(type);
    if (other != ScalarType::Undefined) want += std::string(" or ") + c10::toString(other);
    want += " tensor of shape [";
    const char *comma = "";
    for (const int64_t n : shape) want += comma + (n < 0 ? std::string("*") : std::to_string(n)), comma = ", ";
    want += "] on " + device.str() + ", contiguous" + (strided ? " but for the stride of its first dimension" : "");
    throw BadTensor(want);
}

// The call's device, made the current one for it, and its stream.
struct Launch {
    c10::Device device;
    c10::cuda::OptionalCUDAGuard guard;
    void *stream;

    Launch(const Tensor &t, PyObject *of) : device(t.device()) {
        if (!device.is_cuda()) throw BadTensor("the tensors must be CUDA tensors");
        guard.set_device(device);
        if (of == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
        } else {
            stream = PyLong_AsVoidPtr(of);
            if (PyErr_Occurred()) throw BadTensor("stream must be None or a stream's address");
        }
    }
};

int int_of(PyObject *obj, const char *name) {
    const long x = PyLong_AsLong(obj);
    if (PyErr_Occurred() || x != (long)(int)x) {
        PyErr_Clear();
        throw BadTensor(std::string(name) + " must be a 32-bit integer");
    }
    return (int)x;
}

int *i32(const Tensor &t) { return static_cast<int *>(t.data_ptr()); }
float *f32(const Tensor &t) { return static_cast<float *>(t.data_ptr()); }
int size(const Tensor &t, int64_t d) {
    const int64_t n = t.size(d);
    if (n > 0x7fffffff) throw BadTensor("a tensor's size is out of range");
    return (int)n;
}
// Elements between tokens of a [T, H, D] tensor (one token: its own size).
long long token_stride(const Tensor &t) { return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2); }

template <class F>
PyObject *call(Py_ssize_t given, Py_ssize_t wanted, F f) {
    if (given != wanted) {
        PyErr_Format(PyExc_TypeError, "%zd arguments are wanted, not %zd", wanted, given);
        return nullptr;
    }
    try {
        return PyLong_FromLong(f());
    } catch (const BadTensor &e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception &e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// The C call without the interpreter's lock, as ctypes makes its calls.  The lock is
// taken back by a destructor: a tensor without storage throws when it is asked for
// its address, and the exception has to leave with the lock held.
template <class F>
int unlocked(F f) {
    struct Unlock {
        PyThreadState *const state = PyEval_SaveThread();
        ~Unlock() { PyEval_RestoreThread(state); }
    } unlock;
    return f();
}

// cached_lens, new_lens, free_pages, free_count, block_table, num_pages, page_size, cu_q, seq_lens, slot_map, free_left, positions, stream
PyObject *kv_plan(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call(n, 13, [&] {
        const Tensor &cached = tensor_of(a[0], "cached_lens"), &fresh = tensor_of(a[1], "new_lens");
        const Tensor &free_pages = tensor_of(a[2], "free_pages"), &count = tensor_of(a[3], "free_count");
        const Tensor &table = tensor_of(a[4], "block_table"), &cu = tensor_of(a[7], "cu_q"), &lens = tensor_of(a[8], "seq_lens");
        const Tensor &slots = tensor_of(a[9], "slot_map"), &left = tensor_of(a[10], "free_left");
        const Tensor *positions = tensor_or_none(a[11], "positions");
        Launch at(cached, a[12]);
        const ScalarType i = ScalarType::Int;
        check("cached_lens", cached, at.device, i, {-1});
        const int B = size(cached, 0);
        check("new_lens", fresh, at.device, i, {B});
        check("free_pages", free_pages, at.device, i, {-1});
        check("free_count", count, at.device, i, {1});
        check("block_table", table, at.device, i, {B, -1});
        check("cu_q", cu, at.device, i, {(int64_t)B + 1});
        check("seq_lens", lens, at.device, i, {B});
        check("slot_map", slots, at.device, i, {-1});
        check("free_left", left, at.device, i, {1});
        const int num_pages = int_of(a[5], "num_pages"), page = int_of(a[6], "page_size");
        const int T = size(slots, 0), width = size(table, 1), num_free = size(free_pages, 0);
        if (positions) check("positions", *positions, at.device, i, {T});
        return unlocked([&] {
            if (positions)
                return fa_kv_plan_positions(i32(cached), i32(fresh), i32(free_pages), i32(count), i32(table), i32(cu), i32(lens), i32(slots),
                                            i32(*positions), i32(left), B, T, width, num_free, num_pages, page, at.stream);
            return fa_kv_plan(i32(cached), i32(fresh), i32(free_pages), i32(count), i32(table), i32(cu), i32(lens), i32(slots), i32(left), B, T,
                              width, num_free, num_pages, page, at.stream);
        });
    });
}

struct Cache {
    int num_pages, Hkv, page, D;
};

Cache check_cache(const Tensor &kp, const Tensor &vp, const Tensor &ks, const Tensor &vs, c10::Device device) {
    if (kp.dim() != 4) throw BadTensor("k_pages must be [num_pages, Hkv, page_size, D]");
    const Cache c{size(kp, 0), size(kp, 1), size(kp, 2), size(kp, 3)};
    check("k_pages", kp, device, ScalarType::Byte, {c.num_pages, c.Hkv, c.page, c.D}, false, ScalarType::Float8_e4m3fn);
    check("v_pages", vp, device, ScalarType::Byte, {c.num_pages, c.Hkv, c.page, c.D}, false, ScalarType::Float8_e4m3fn);
    check("k_scale", ks, device, ScalarType::Float, {c.num_pages, c.Hkv});
    check("v_scale", vs, device, ScalarType::Float, {c.num_pages, c.Hkv});
    return c;
}

// k, v, slot_map, k_pages, v_pages, k_scale, v_scale, k_mean, k_mean_scale, stream
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call(n, 10, [&] {
        const Tensor &k = tensor_of(a[0], "k"), &v = tensor_of(a[1], "v"), &slots = tensor_of(a[2], "slot_map");
        const Tensor &kp = tensor_of(a[3], "k_pages"), &vp = tensor_of(a[4], "v_pages");
        const Tensor &ks = tensor_of(a[5], "k_scale"), &vs = tensor_of(a[6], "v_scale");
        const Tensor *mean = tensor_or_none(a[7], "k_mean"), *mean_scale = tensor_or_none(a[8], "k_mean_scale");
        Launch at(k, a[9]);
        const Cache c = check_cache(kp, vp, ks, vs, at.device);
        check("slot_map", slots, at.device, ScalarType::Int, {-1});
        const int T = size(slots, 0);
        check("k", k, at.device, ScalarType::BFloat16, {T, c.Hkv, c.D}, true);
        check("v", v, at.device, ScalarType::BFloat16, {T, c.Hkv, c.D}, true);
        if (!mean != !mean_scale) throw BadTensor("give both of k_mean and k_mean_scale, or neither");
        if (mean) {
            check("k_mean", *mean, at.device, ScalarType::Char, {c.num_pages, c.Hkv, c.D});
            check("k_mean_scale", *mean_scale, at.device, ScalarType::Float, {c.num_pages, c.Hkv});
        }
        return unlocked([&] {
            return fa_kv_append(k.data_ptr(), v.data_ptr(), i32(slots), kp.data_ptr(), vp.data_ptr(), f32(ks), f32(vs),
                                mean ? static_cast<signed char *>(mean->data_ptr()) : nullptr, mean ? f32(*mean_scale) : nullptr, T, c.Hkv, c.D,
                                token_stride(k), token_stride(v), c.num_pages, c.page, at.stream);
        });
    });
}

// What a rotation is made of: phases, interleaved, amplitude.
struct Rotation {
    const unsigned long long *phases;
    int rot_dim, interleaved;
    float amplitude;
};

float float_of(PyObject *obj, const char *name) {
    const double x = PyFloat_AsDouble(obj);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        throw BadTensor(std::string(name) + " must be a number");
    }
    return (float)x;
}

Rotation rotation_of(PyObject *phases, PyObject *interleaved, PyObject *amplitude, c10::Device device) {
    const Tensor &t = tensor_of(phases, "phases");
    check("phases", t, device, ScalarType::Long, {-1});
    if (t.size(0) > 64) throw BadTensor("phases must be of one element for each pair of a head's elements");
    const int i = PyObject_IsTrue(interleaved);
    if (i < 0) {
        PyErr_Clear();
        throw BadTensor("interleaved must be a truth value");
    }
    return Rotation{reinterpret_cast<const unsigned long long *>(t.data_ptr()), 2 * (int)t.size(0), i, float_of(amplitude, "amplitude")};
}

// k, v, positions, phases, slot_map, k_pages, v_pages, k_scale, v_scale, k_mean, k_mean_scale, q, q_out, interleaved, amplitude, stream
PyObject *kv_append_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call(n, 16, [&] {
        const Tensor &k = tensor_of(a[0], "k"), &v = tensor_of(a[1], "v"), &positions = tensor_of(a[2], "positions");
        const Tensor &slots = tensor_of(a[4], "slot_map"), &kp = tensor_of(a[5], "k_pages"), &vp = tensor_of(a[6], "v_pages");
        const Tensor &ks = tensor_of(a[7], "k_scale"), &vs = tensor_of(a[8], "v_scale");
        const Tensor *mean = tensor_or_none(a[9], "k_mean"), *mean_scale = tensor_or_none(a[10], "k_mean_scale");
        const Tensor *q = tensor_or_none(a[11], "q"), *q_out = tensor_or_none(a[12], "q_out");
        Launch at(k, a[15]);
        const Rotation r = rotation_of(a[3], a[13], a[14], at.device);
        const Cache c = check_cache(kp, vp, ks, vs, at.device);
        check("slot_map", slots, at.device, ScalarType::Int, {-1});
        const int T = size(slots, 0);
        check("positions", positions, at.device, ScalarType::Int, {T});
        check("k", k, at.device, ScalarType::BFloat16, {T, c.Hkv, c.D}, true);
        check("v", v, at.device, ScalarType::BFloat16, {T, c.Hkv, c.D}, true);
        if (!mean != !mean_scale) throw BadTensor("give both of k_mean and k_mean_scale, or neither");
        if (mean) {
            check("k_mean", *mean, at.device, ScalarType::Char, {c.num_pages, c.Hkv, c.D});
            check("k_mean_scale", *mean_scale, at.device, ScalarType::Float, {c.num_pages, c.Hkv});
        }
        if (!q != !q_out) throw BadTensor("give both of q and q_out, or neither");
        int Hq = 0;
        if (q) {
            check("q", *q, at.device, ScalarType::BFloat16, {T, -1, c.D}, true);
            Hq = size(*q, 1);
            check("q_out", *q_out, at.device, ScalarType::BFloat16, {T, Hq, c.D}, true);
        }
        return unlocked([&] {
            return fa_kv_append_rope(k.data_ptr(), v.data_ptr(), i32(positions), r.phases, i32(slots), kp.data_ptr(), vp.data_ptr(), f32(ks),
                                     f32(vs), mean ? static_cast<signed char *>(mean->data_ptr()) : nullptr, mean ? f32(*mean_scale) : nullptr,
                                     q ? q->data_ptr() : nullptr, q ? q_out->data_ptr() : nullptr, T, c.Hkv, Hq, c.D, r.rot_dim, r.interleaved,
                                     r.amplitude, token_stride(k), token_stride(v), q ? token_stride(*q) : 0, q ? token_stride(*q_out) : 0,
                                     c.num_pages, c.page, at.stream);
        });
    });
}

// A tensor [T, H, D] or [B, H, S, D] that a rotation reads or writes: its strides between
// sequences, tokens and heads.  (A dimension of size 1 has no stride that counts.)
void rope_strides(const char *name, const Tensor &t, const Tensor &like, bool heads, c10::Device device, long long *strides) {
    const int64_t d = t.dim();
    const bool fits = t.scalar_type() == ScalarType::BFloat16 && t.device() == device && d == like.dim() && t.size(d - 1) == like.size(d - 1) &&
                      t.stride(d - 1) == 1 && t.size(d - 3 + (d == 3 ? 0 : 1)) == like.size(d - 3 + (d == 3 ? 0 : 1)) &&
                      (d == 3 || t.size(0) == like.size(0)) && (!heads || t.size(1) == like.size(1));
    if (!fits)
        throw BadTensor(std::string(name) + " must be a BFloat16 tensor [T, H, D] or [B, H, S, D] on " + device.str() +
                        " whose last dimension is contiguous, of the other tensors' sizes");
    const auto stride = [&](int64_t i) -> long long { return t.size(i) > 1 ? t.stride(i) : 0; };
    if (d == 3)
        strides[0] = 0, strides[1] = stride(0), strides[2] = stride(1);
    else
        strides[0] = stride(0), strides[1] = stride(2), strides[2] = stride(1);
}

// q, k, phases, positions, interleaved, amplitude, q_out, k_out, inverse, stream
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call(n, 10, [&] {
        const Tensor &q = tensor_of(a[0], "q"), &q_out = tensor_of(a[6], "q_out");
        const Tensor *k = tensor_or_none(a[1], "k"), *k_out = tensor_or_none(a[7], "k_out"), *positions = tensor_or_none(a[3], "positions");
        Launch at(q, a[9]);
        const Rotation r = rotation_of(a[2], a[4], a[5], at.device);
        if (q.dim() != 3 && q.dim() != 4) throw BadTensor("q must be [T, H, D] or [B, H, S, D]");
        if (!k != !k_out) throw BadTensor("give both of k and k_out, or neither");
        long long strides[12] = {};
        rope_strides("q", q, q, true, at.device, strides);
        rope_strides("q_out", q_out, q, true, at.device, strides + 6);
        if (k) {
            rope_strides("k", *k, q, false, at.device, strides + 3);
            rope_strides("k_out", *k_out, *k, true, at.device, strides + 9);
        }
        const bool packed = q.dim() == 3;
        const int B = packed ? 1 : size(q, 0), S = packed ? size(q, 0) : size(q, 2);
        long long positions_stride = 0;
        if (positions && positions->dim() == 2 && !packed) {
            check("positions", *positions, at.device, ScalarType::Int, {B, S});
            positions_stride = S;
        } else if (positions) {
            check("positions", *positions, at.device, ScalarType::Int, {S});
        }
        const bool inverse = PyObject_IsTrue(a[8]) == 1;
        return unlocked([&] {
            return (inverse ? fa_rope_bwd : fa_rope)(q.data_ptr(), k ? k->data_ptr() : nullptr, q_out.data_ptr(), k ? k_out->data_ptr() : nullptr,
                                                     positions ? i32(*positions) : nullptr, r.phases, B, S, size(q, 1), k ? size(*k, 1) : 0,
                                                     size(q, q.dim() - 1), r.rot_dim, strides, positions_stride, r.interleaved, r.amplitude,
                                                     at.stream);
        });
    });
}

struct Queries {
    int B, T, Hq, width;
};

Queries check_queries(const Tensor &q, const Tensor &cu, const Tensor &lens, const Tensor &table, int D, c10::Device device) {
    check("q", q, device, ScalarType::BFloat16, {-1, -1, D}, true);
    check("seq_lens", lens, device, ScalarType::Int, {-1});
    const int64_t B = lens.size(0);
    check("cu_q", cu, device, ScalarType::Int, {B + 1});
    check("block_table", table, device, ScalarType::Int, {B, -1});
    return Queries{size(lens, 0), size(q, 0), size(q, 1), size(table, 1)};
}

// q, cu_q, seq_lens, block_table, k_mean, k_mean_scale, page_size, top_k, keep_first, keep_last, sel, sel_count, stream
PyObject *page_select(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call(n, 13, [&] {
        const Tensor &q = tensor_of(a[0], "q"), &cu = tensor_of(a[1], "cu_q"), &lens = tensor_of(a[2], "seq_lens");
        const Tensor &table = tensor_of(a[3], "block_table"), &mean = tensor_of(a[4], "k_mean"), &ms = tensor_of(a[5], "k_mean_scale");
        const Tensor &sel = tensor_of(a[10], "sel"), &count = tensor_of(a[11], "sel_count");
        Launch at(q, a[12]);
        check("k_mean", mean, at.device, ScalarType::Char, {-1, -1, -1});
        const int num_pages = size(mean, 0), Hkv = size(mean, 1), D = size(mean, 2);
        check("k_mean_scale", ms, at.device, ScalarType::Float, {num_pages, Hkv});
        const Queries s = check_queries(q, cu, lens, table, D, at.device);
        const int page = int_of(a[6], "page_size"), top_k = int_of(a[7], "top_k");
        const int first = int_of(a[8], "keep_first"), last = int_of(a[9], "keep_last");
        check("sel", sel, at.device, ScalarType::Int, {s.B, Hkv, top_k});
        check("sel_count", count, at.device, ScalarType::Int, {s.B, Hkv});
        return unlocked([&] {
            return fa_page_select(q.data_ptr(), i32(cu), i32(lens), i32(table), static_cast<signed char *>(mean.data_ptr()), f32(ms), i32(sel),
                                  i32(count), s.B, s.T, s.Hq, Hkv, D, token_stride(q), s.width, num_pages, page, top_k, first, last, at.stream);
        });
    });
}

// q, cu_q, seq_lens, block_table, k_pages, v_pages, k_scale, v_scale, sel, sel_count, o, lse, scale, workspace, stream
PyObject *fwd_paged(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call(n, 15, [&] {
        const Tensor &q = tensor_of(a[0], "q"), &cu = tensor_of(a[1], "cu_q"), &lens = tensor_of(a[2], "seq_lens");
        const Tensor &table = tensor_of(a[3], "block_table"), &kp = tensor_of(a[4], "k_pages"), &vp = tensor_of(a[5], "v_pages");
        const Tensor &ks = tensor_of(a[6], "k_scale"), &vs = tensor_of(a[7], "v_scale");
        const Tensor *sel = tensor_or_none(a[8], "sel"), *count = tensor_or_none(a[9], "sel_count");
        const Tensor &o = tensor_of(a[10], "o"), &lse = tensor_of(a[11], "lse"), &ws = tensor_of(a[13], "workspace");
        const float scale = float_of(a[12], "scale");
        Launch at(q, a[14]);
        const Cache c = check_cache(kp, vp, ks, vs, at.device);
        const Queries s = check_queries(q, cu, lens, table, c.D, at.device);
        if (!sel != !count) throw BadTensor("give both of sel and sel_count, or neither");
        if (sel) {
            check("sel", *sel, at.device, ScalarType::Int, {s.B, c.Hkv, -1});
            check("sel_count", *count, at.device, ScalarType::Int, {s.B, c.Hkv});
        }
        check("o", o, at.device, ScalarType::BFloat16, {s.T, s.Hq, c.D});
        check("lse", lse, at.device, ScalarType::Float, {s.T, s.Hq});
        check("workspace", ws, at.device, ScalarType::Byte, {-1});
        return unlocked([&] {
            return fa_fwd_paged(q.data_ptr(), i32(cu), i32(lens), i32(table), kp.data_ptr(), vp.data_ptr(), f32(ks), f32(vs),
                                sel ? i32(*sel) : nullptr, sel ? i32(*count) : nullptr, o.data_ptr(), f32(lse), s.B, s.T, s.Hq, c.Hkv, c.D,
                                scale, token_stride(q), s.width, c.num_pages, c.page, sel ? size(*sel, 2) : 0, ws.data_ptr(),
                                (size_t)ws.numel(), at.stream);
        });
    });
}

// q, cu_q, seq_lens, block_table, k_pages, v_pages, k_scale, v_scale, o, lse, scale, workspace, stream
PyObject *fwd_paged_chunk(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call(n, 13, [&] {
        const Tensor &q = tensor_of(a[0], "q"), &cu = tensor_of(a[1], "cu_q"), &lens = tensor_of(a[2], "seq_lens");
        const Tensor &table = tensor_of(a[3], "block_table"), &kp = tensor_of(a[4], "k_pages"), &vp = tensor_of(a[5], "v_pages");
        const Tensor &ks = tensor_of(a[6], "k_scale"), &vs = tensor_of(a[7], "v_scale");
        const Tensor &o = tensor_of(a[8], "o"), &lse = tensor_of(a[9], "lse"), &ws = tensor_of(a[11], "workspace");
        const float scale = float_of(a[10], "scale");
        Launch at(q, a[12]);
        const Cache c = check_cache(kp, vp, ks, vs, at.device);
        const Queries s = check_queries(q, cu, lens, table, c.D, at.device);
        check("o", o, at.device, ScalarType::BFloat16, {s.T, s.Hq, c.D});
        check("lse", lse, at.device, ScalarType::Float, {s.T, s.Hq});
        check("workspace", ws, at.device, ScalarType::Byte, {-1});
        return unlocked([&] {
            return fa_fwd_paged_chunk(q.data_ptr(), i32(cu), i32(lens), i32(table), kp.data_ptr(), vp.data_ptr(), f32(ks), f32(vs), o.data_ptr(),
                                      f32(lse), s.B, s.T, s.Hq, c.Hkv, c.D, scale, token_stride(q), s.width, c.num_pages, c.page, ws.data_ptr(),
                                      (size_t)ws.numel(), at.stream);
        });
    });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"kv_plan", FAST(kv_plan), "fa_kv_plan on tensors"},
                         {"kv_append", FAST(kv_append), "fa_kv_append on tensors"},
                         {"page_select", FAST(page_select), "fa_page_select on tensors"},
                         {"fwd_paged", FAST(fwd_paged), "fa_fwd_paged on tensors"},
                         {"fwd_paged_chunk", FAST(fwd_paged_chunk), "fa_fwd_paged_chunk on tensors"},
                         {"kv_append_rope", FAST(kv_append_rope), "fa_kv_append_rope on tensors"},
                         {"rope", FAST(rope), "fa_rope and fa_rope_bwd on tensors"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "fa_binding", "The paged cache's calls for torch tensors.", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fa_binding() { return PyModule_Create(&module); }

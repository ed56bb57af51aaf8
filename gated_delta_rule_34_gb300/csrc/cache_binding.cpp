// The global-attention operators' calls from Python.
//
// A decode step's kernels take 3 to 17 us.  With the checks in Python, the C entry through ctypes (25 arguments) and a
// torch.empty for each result the host spent more than that on a call.  Here a call reads the tensors' sizes,
// strides and addresses directly, allocates through ATen and calls the C entry.  Host time of a call, in a loop of
// them: rotary of a token 5.3 us (16 to 18 through Python), a token written for each of 256 sequences 4.0 (13 to 14),
// attention of a short sequence 6.6 (18 to 21).
//
// What is well formed is launched; for anything else a function returns None and launches nothing, and its caller in
// cache.py, which knows the arguments' names, says what is wrong.  The library's own refusals come back as its status and are
// raised by api._check.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <cmath>

#include "kda.h"

namespace {

// The entries of the library that ctypes has loaded, so that there is one copy of it in the process.
decltype(&kda_rotary) rotary_entry;
decltype(&kda_cache_write) write_entry;
decltype(&kda_cache_read) read_entry;
decltype(&kda_cache_attention) attention_entry;
decltype(&kda_cache_attention_workspace_size) workspace_entry;
decltype(&kda_cache_copy) copy_entry;
decltype(&kda_cache_resize) resize_entry;
decltype(&kda_cache_fork) fork_entry;
decltype(&kda_cache_compact) compact_entry;
decltype(&kda_cache_pages_workspace_size) pages_workspace_entry;
decltype(&kda_cache_attention_shared) shared_entry;
decltype(&kda_cache_attention_shared_workspace_size) shared_workspace_entry;
PyObject* check;                           // api._check

const at::Tensor* tensor(PyObject* x) { return THPVariable_Check(x) ? &THPVariable_Unpack(x) : nullptr; }

// The current device's index where t is on it, else -1.
int current_device_of(const at::Tensor* t) {
    if (!t || !t->is_cuda()) return -1;
    const int index = t->get_device();
    return index == c10::cuda::current_device() ? index : -1;
}

bool dense(const at::Tensor* t, at::ScalarType type, int index) {
    return t && t->is_cuda() && t->get_device() == index && t->scalar_type() == type && t->is_contiguous();
}
bool dense(const at::Tensor* t, at::ScalarType type, int index, at::IntArrayRef shape) {
    return dense(t, type, index) && t->sizes() == shape;
}

bool code_of(at::ScalarType type, kda_dtype& code) {
    code = type == at::kFloat ? KDA_DTYPE_F32 : KDA_DTYPE_BF16;
    return type == at::kFloat || type == at::kBFloat16;
}

// The token stride of [..., tokens, H, d] whose [H, d] are dense and whose tokens are evenly spaced, else -1.
int64_t token_stride(const at::Tensor* t, at::ScalarType type, int index) {
    if (!t || !t->is_cuda() || t->get_device() != index || t->scalar_type() != type || t->dim() < 3) return -1;
    const int64_t n = t->dim(), h = t->size(n - 2), d = t->size(n - 1);
    if (t->is_contiguous()) return h * d;
    if ((d > 1 && t->stride(n - 1) != 1) || (h > 1 && t->stride(n - 2) != d)) return -1;
    int64_t stride = -1, span = 0;
    for (int64_t i = n - 3; i >= 0; --i) {
        if (t->size(i) == 1) continue;
        if (stride < 0) {
            stride = t->stride(i);
            span = stride * t->size(i);
        } else if (t->stride(i) != span) {
            return -1;
        } else {
            span *= t->size(i);
        }
    }
    return stride < 0 ? h * d : stride < h * d ? -1 : stride;
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}

struct Pool {
    const at::Tensor *k, *v, *k_scale, *v_scale;
    int64_t n_pages, h, page, d;

    bool read(PyObject* cache, int index) {
        return PyTuple_Check(cache) && PyTuple_GET_SIZE(cache) == 4 && (k = tensor(PyTuple_GET_ITEM(cache, 0))) &&
               (v = tensor(PyTuple_GET_ITEM(cache, 1))) && (k_scale = tensor(PyTuple_GET_ITEM(cache, 2))) &&
               (v_scale = tensor(PyTuple_GET_ITEM(cache, 3))) && k->dim() == 4 &&
               dense(k, at::kFloat8_e4m3fn, index) && dense(v, at::kFloat8_e4m3fn, index, k->sizes()) &&
               dense(k_scale, at::kFloat, index, k->sizes().slice(0, 2)) &&
               dense(v_scale, at::kFloat, index, k->sizes().slice(0, 2)) && sizes();
    }
    bool sizes() {
        n_pages = k->size(0), h = k->size(1), page = k->size(2), d = k->size(3);
        return h <= INT_MAX && page <= INT_MAX && d <= INT_MAX;
    }
};

// The sequences of packed or batched rows with their block table and starts.
struct Sequences {
    const at::Tensor *table, *start, *cu;
    int64_t n;

    bool read(int64_t batch, PyObject* cu_obj, PyObject* table_obj, PyObject* start_obj, int index) {
        table = tensor(table_obj);
        start = tensor(start_obj);
        cu = tensor(cu_obj);
        n = batch;
        if (cu_obj != Py_None) {
            if (!cu || batch != 1 || cu->dim() != 1 || cu->numel() < 1 || !dense(cu, at::kInt, index)) return false;
            n = cu->numel() - 1;
        }
        return n <= INT_MAX && dense(table, at::kInt, index) && table->dim() == 2 && table->size(0) == n &&
               table->size(1) <= INT_MAX && dense(start, at::kInt, index, {n});
    }
    const int32_t* cu_ptr() const { return cu ? cu->const_data_ptr<int32_t>() : nullptr; }
};

bool failed(kda_status status) {
    if (status == KDA_OK) return false;
    Py_XDECREF(PyObject_CallFunction(check, "i", (int)status));
    return true;
}

// Integers as the C entries take them; false with an error set.
bool integer(PyObject* x, int64_t& to) {
    to = PyLong_AsLongLong(x);
    return !(to == -1 && PyErr_Occurred());
}
bool integer32(PyObject* x, int& to) {
    int64_t wide;
    if (!integer(x, wide)) return false;
    to = (int)wide;
    if (to == wide) return true;
    PyErr_SetString(PyExc_OverflowError, "an argument does not fit into 32 bits");
    return false;
}
bool real(PyObject* x, float& to) {
    const double wide = PyFloat_AsDouble(x);
    to = (float)wide;
    return !(wide == -1.0 && PyErr_Occurred());
}

PyObject* pair_of(PyObject* a, PyObject* b) {
    PyObject* t = a && b ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return t;
}
// What was given, or what was allocated in its place.
PyObject* result(PyObject* given, const at::Tensor& made) {
    return given == Py_None ? THPVariable_Wrap(made) : Py_NewRef(given);
}

bool takes(const char* name, Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, n);
    return false;
}

// q, k, positions, freq, layout, amplitude, q_out, k_out -> (q_out, k_out)
PyObject* rotary(PyObject*, PyObject* const* arg, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    if (!takes("rotary", n_args, 8)) return nullptr;
    const at::Tensor *q = tensor(arg[0]), *k = tensor(arg[1]), *positions = tensor(arg[2]), *freq = tensor(arg[3]);
    const int index = current_device_of(q);
    kda_dtype code;
    if (index < 0 || !code_of(q->scalar_type(), code)) Py_RETURN_NONE;
    const at::ScalarType type = q->scalar_type();
    const int64_t q_stride = token_stride(q, type, index);
    if (q_stride < 0) Py_RETURN_NONE;
    const int64_t dims = q->dim(), h_q = q->size(dims - 2), d = q->size(dims - 1);
    const int64_t n = h_q > 0 && d > 0 ? q->numel() / (h_q * d) : 0;
    int64_t k_stride = 0, h_k = 0;
    if (arg[1] != Py_None) {
        if (!k || (k_stride = token_stride(k, type, index)) < 0 || k->dim() != dims || k->size(dims - 1) != d ||
            k->sizes().slice(0, dims - 2) != q->sizes().slice(0, dims - 2))
            Py_RETURN_NONE;
        h_k = k->size(dims - 2);
    } else if (arg[7] != Py_None) {
        Py_RETURN_NONE;
    }
    if (!dense(positions, at::kInt, index) || positions->numel() != n || !dense(freq, at::kDouble, index) ||
        freq->dim() != 1 || h_q > INT_MAX || h_k > INT_MAX || d > INT_MAX || 2 * freq->numel() > INT_MAX)
        Py_RETURN_NONE;
    kda_rotary_layout layout;
    if (!PyUnicode_Check(arg[4])) Py_RETURN_NONE;
    if (PyUnicode_CompareWithASCIIString(arg[4], "half") == 0) layout = KDA_ROTARY_HALF;
    else if (PyUnicode_CompareWithASCIIString(arg[4], "interleaved") == 0) layout = KDA_ROTARY_INTERLEAVED;
    else Py_RETURN_NONE;
    float amplitude;
    if (!real(arg[5], amplitude)) return nullptr;
    at::Tensor q_made, k_made;
    const at::Tensor *q_out = &q_made, *k_out = &k_made;
    int64_t qo_stride = h_q * d, ko_stride = h_k * d;
    if (arg[6] != Py_None) {
        q_out = tensor(arg[6]);
        if (!q_out || (qo_stride = token_stride(q_out, type, index)) < 0 || q_out->sizes() != q->sizes()) Py_RETURN_NONE;
    }
    if (arg[7] != Py_None) {
        k_out = tensor(arg[7]);
        if (!k_out || (ko_stride = token_stride(k_out, type, index)) < 0 || k_out->sizes() != k->sizes()) Py_RETURN_NONE;
    }
    if (arg[6] == Py_None) q_made = empty(q->sizes(), type, *q);
    if (k && arg[7] == Py_None) k_made = empty(k->sizes(), type, *q);
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(index).stream();
    kda_status status;
    Py_BEGIN_ALLOW_THREADS
    status = rotary_entry(q->const_data_ptr(), q_stride, q_out->mutable_data_ptr(), qo_stride, (int)h_q,
                          k ? k->const_data_ptr() : nullptr, k_stride, k ? k_out->mutable_data_ptr() : nullptr,
                          k ? ko_stride : 0, (int)h_k, positions->const_data_ptr<int32_t>(),
                          freq->const_data_ptr<double>(), amplitude, n, (int)d, (int)(2 * freq->numel()), layout, code,
                          stream);
    Py_END_ALLOW_THREADS
    if (failed(status)) return nullptr;
    return pair_of(result(arg[6], q_made), k ? result(arg[7], k_made) : Py_NewRef(Py_None));
    END_HANDLE_TH_ERRORS
}

// cache, k, v, block_table, start, cu_seqlens -> cache
PyObject* cache_write(PyObject*, PyObject* const* arg, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    if (!takes("cache_write", n_args, 6)) return nullptr;
    const at::Tensor *k = tensor(arg[1]), *v = tensor(arg[2]);
    const int index = current_device_of(k);
    kda_dtype code;
    if (index < 0 || !code_of(k->scalar_type(), code)) Py_RETURN_NONE;
    const int64_t k_stride = token_stride(k, k->scalar_type(), index);
    const int64_t v_stride = token_stride(v, k->scalar_type(), index);
    Pool pool;
    Sequences seqs;
    if (k_stride < 0 || v_stride < 0 || !pool.read(arg[0], index) || k->dim() != 4 || v->sizes() != k->sizes() ||
        k->size(2) != pool.h || k->size(3) != pool.d || !seqs.read(k->size(0), arg[5], arg[3], arg[4], index))
        Py_RETURN_NONE;
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(index).stream();
    kda_status status;
    Py_BEGIN_ALLOW_THREADS
    status = write_entry(k->const_data_ptr(), k_stride, v->const_data_ptr(), v_stride, pool.k->mutable_data_ptr(),
                         pool.v->mutable_data_ptr(), pool.k_scale->mutable_data_ptr<float>(),
                         pool.v_scale->mutable_data_ptr<float>(), seqs.table->const_data_ptr<int32_t>(),
                         (int)seqs.table->size(1), seqs.start->const_data_ptr<int32_t>(), seqs.cu_ptr(), (int)seqs.n,
                         k->size(1), (int)pool.h, (int)pool.d, pool.n_pages, (int)pool.page, code, stream);
    Py_END_ALLOW_THREADS
    if (failed(status)) return nullptr;
    return Py_NewRef(arg[0]);
    END_HANDLE_TH_ERRORS
}

// cache, block_table, start, T, cu_seqlens, dtype, k_out, v_out -> (k, v)
PyObject* cache_read(PyObject*, PyObject* const* arg, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    if (!takes("cache_read", n_args, 8)) return nullptr;
    if (!PyTuple_Check(arg[0]) || PyTuple_GET_SIZE(arg[0]) != 4 || !THPDtype_Check(arg[5])) Py_RETURN_NONE;
    const int index = current_device_of(tensor(PyTuple_GET_ITEM(arg[0], 0)));
    const at::ScalarType type = reinterpret_cast<THPDtype*>(arg[5])->scalar_type;
    const at::Tensor* table = tensor(arg[1]);
    const bool packed = arg[4] != Py_None;
    Pool pool;
    Sequences seqs;
    kda_dtype code;
    if (index < 0 || !code_of(type, code) || !pool.read(arg[0], index) || !table || table->dim() != 2 ||
        !seqs.read(packed ? 1 : table->size(0), arg[4], arg[1], arg[2], index))
        Py_RETURN_NONE;
    int64_t t;
    if (!integer(arg[3], t)) return nullptr;
    const int64_t shape[4] = {packed ? 1 : seqs.n, t, pool.h, pool.d};
    at::Tensor k_made, v_made;
    const at::Tensor *k = &k_made, *v = &v_made;
    if (arg[6] != Py_None && !dense(k = tensor(arg[6]), type, index, shape)) Py_RETURN_NONE;
    if (arg[7] != Py_None && !dense(v = tensor(arg[7]), type, index, shape)) Py_RETURN_NONE;
    if (arg[6] == Py_None) k_made = empty(shape, type, *pool.k);
    if (arg[7] == Py_None) v_made = empty(shape, type, *pool.k);
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(index).stream();
    kda_status status;
    Py_BEGIN_ALLOW_THREADS
    status = read_entry(pool.k->const_data_ptr(), pool.v->const_data_ptr(), pool.k_scale->const_data_ptr<float>(),
                        pool.v_scale->const_data_ptr<float>(), seqs.table->const_data_ptr<int32_t>(),
                        (int)seqs.table->size(1), seqs.start->const_data_ptr<int32_t>(), seqs.cu_ptr(), (int)seqs.n, t,
                        (int)pool.h, (int)pool.d, pool.n_pages, (int)pool.page, k->mutable_data_ptr(),
                        v->mutable_data_ptr(), code, stream);
    Py_END_ALLOW_THREADS
    if (failed(status)) return nullptr;
    return pair_of(result(arg[6], k_made), result(arg[7], v_made));
    END_HANDLE_TH_ERRORS
}

// q, cache, block_table, lengths, scale, window, sinks, out, lse, return_lse, workspace -> o or (o, lse)
PyObject* cache_attention(PyObject*, PyObject* const* arg, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    if (!takes("cache_attention", n_args, 11)) return nullptr;
    const at::Tensor *q = tensor(arg[0]), *table = tensor(arg[2]), *lengths = tensor(arg[3]);
    const int index = current_device_of(q);
    kda_dtype code;
    if (index < 0 || !code_of(q->scalar_type(), code) || q->dim() != 4) Py_RETURN_NONE;
    const at::ScalarType type = q->scalar_type();
    const int64_t q_stride = token_stride(q, type, index);
    Pool pool;
    if (q_stride < 0 || !pool.read(arg[1], index) || q->size(3) != pool.d) Py_RETURN_NONE;
    const int64_t B = q->size(0), t_q = q->size(1), h_q = q->size(2);
    if (!dense(table, at::kInt, index) || table->dim() != 2 || table->size(0) != B || !dense(lengths, at::kInt, index, {B}) ||
        B > INT_MAX || t_q > INT_MAX || h_q > INT_MAX || table->size(1) > INT_MAX)
        Py_RETURN_NONE;
    const int wide = (int)table->size(1), d = (int)pool.d;
    float scale = (float)(1.0 / std::sqrt((double)d));
    int64_t window;
    int sinks;
    if ((arg[4] != Py_None && !real(arg[4], scale)) || !integer(arg[5], window) || !integer32(arg[6], sinks)) return nullptr;
    const int with_lse = PyObject_IsTrue(arg[9]);
    if (with_lse < 0) return nullptr;

    at::Tensor o_made, lse_made, ws_made;
    const at::Tensor *o = &o_made, *lse = arg[8] != Py_None ? tensor(arg[8]) : with_lse ? &lse_made : nullptr, *ws = &ws_made;
    if (arg[7] != Py_None && !dense(o = tensor(arg[7]), type, index, q->sizes())) Py_RETURN_NONE;
    if (arg[8] != Py_None && !dense(lse, at::kFloat, index, q->sizes().slice(0, 3))) Py_RETURN_NONE;
    if (arg[10] != Py_None) {
        ws = tensor(arg[10]);
        if (!ws || !ws->is_cuda() || ws->get_device() != index || !ws->is_contiguous()) Py_RETURN_NONE;
    }
    if (arg[7] == Py_None) o_made = empty(q->sizes(), type, *q);
    if (lse == &lse_made) lse_made = empty(q->sizes().slice(0, 3), at::kFloat, *q);
    if (arg[10] == Py_None) {
        const size_t need = workspace_entry((int)B, (int)t_q, (int)h_q, (int)pool.h, d, (int)pool.page, wide);
        if (need) ws_made = empty({(int64_t)need}, at::kByte, *q);
    }
    const size_t ws_bytes = ws->defined() ? ws->nbytes() : 0;
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(index).stream();
    kda_status status;
    Py_BEGIN_ALLOW_THREADS
    status = attention_entry(q->const_data_ptr(), q_stride, pool.k->const_data_ptr(), pool.v->const_data_ptr(),
                             pool.k_scale->const_data_ptr<float>(), pool.v_scale->const_data_ptr<float>(),
                             table->const_data_ptr<int32_t>(), wide, lengths->const_data_ptr<int32_t>(),
                             o->mutable_data_ptr(), lse ? lse->mutable_data_ptr<float>() : nullptr, (int)B, (int)t_q,
                             (int)h_q, (int)pool.h, d, pool.n_pages, (int)pool.page, scale, window, sinks, code,
                             ws->defined() ? ws->mutable_data_ptr() : nullptr, ws_bytes, stream);
    Py_END_ALLOW_THREADS
    if (failed(status)) return nullptr;
    PyObject* out = result(arg[7], o_made);
    return with_lse ? pair_of(out, result(arg[8], lse_made)) : out;
    END_HANDLE_TH_ERRORS
}

// cache, src, dst -> cache
PyObject* cache_copy(PyObject*, PyObject* const* arg, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    if (!takes("cache_copy", n_args, 3)) return nullptr;
    const at::Tensor *src = tensor(arg[1]), *dst = tensor(arg[2]);
    const int index = current_device_of(src);
    Pool pool;
    if (index < 0 || !pool.read(arg[0], index) || !dense(src, at::kInt, index) || src->dim() != 1 || src->numel() > INT_MAX ||
        !dense(dst, at::kInt, index, src->sizes()))
        Py_RETURN_NONE;
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(index).stream();
    kda_status status;
    Py_BEGIN_ALLOW_THREADS
    status = copy_entry(pool.k->mutable_data_ptr(), pool.v->mutable_data_ptr(), pool.k_scale->mutable_data_ptr<float>(),
                        pool.v_scale->mutable_data_ptr<float>(), src->const_data_ptr<int32_t>(),
                        dst->const_data_ptr<int32_t>(), (int)src->numel(), (int)pool.h, (int)pool.d, pool.n_pages,
                        (int)pool.page, stream);
    Py_END_ALLOW_THREADS
    if (failed(status)) return nullptr;
    return Py_NewRef(arg[0]);
    END_HANDLE_TH_ERRORS
}

// A dense list of int32, given or to be made; false where what is given is not one.
struct List {
    at::Tensor made;
    const at::Tensor* at = &made;

    bool read(PyObject* given, int64_t n, int index, const at::Tensor& like) {
        if (given == Py_None) {
            made = empty({n}, at::kInt, like);
            return true;
        }
        return dense(at = tensor(given), at::kInt, index, {n});
    }
    int32_t* ptr() const { return at->mutable_data_ptr<int32_t>(); }
};

// The counts and a block table.
struct Rows {
    const at::Tensor *refs, *table;
    int64_t n_pages;

    bool read(PyObject* refs_obj, PyObject* table_obj, int index) {
        refs = tensor(refs_obj);
        table = tensor(table_obj);
        if (!dense(refs, at::kInt, index) || refs->dim() != 1 || !dense(table, at::kInt, index) || table->dim() != 2 ||
            table->size(0) > INT_MAX || table->size(1) > INT_MAX)
            return false;
        n_pages = refs->numel();
        return true;
    }
};

struct Workspace {
    at::Tensor made;
    const at::Tensor* at = &made;

    bool read(PyObject* given, size_t need, int index, const at::Tensor& like) {
        if (given == Py_None) {
            if (need) made = empty({(int64_t)need}, at::kByte, like);
            return true;
        }
        at = tensor(given);
        return at && at->is_cuda() && at->get_device() == index && at->is_contiguous();
    }
    size_t bytes() const { return at->defined() ? at->nbytes() : 0; }
    void* ptr() const { return at->defined() ? at->mutable_data_ptr() : nullptr; }
};

// refs, block_table, rows, tokens, page, missing, workspace -> missing
PyObject* cache_resize(PyObject*, PyObject* const* arg, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    if (!takes("cache_resize", n_args, 7)) return nullptr;
    const at::Tensor *rows = tensor(arg[2]), *tokens = tensor(arg[3]);
    const int index = current_device_of(rows);
    Rows table;
    if (index < 0 || !table.read(arg[0], arg[1], index) || !dense(rows, at::kInt, index) || rows->dim() != 1 ||
        rows->numel() > INT_MAX || !dense(tokens, at::kInt, index, rows->sizes()))
        Py_RETURN_NONE;
    int page;
    if (!integer32(arg[4], page)) return nullptr;
    List missing;
    Workspace ws;
    if (!missing.read(arg[5], 1, index, *rows) || !ws.read(arg[6], pages_workspace_entry(table.n_pages, (int)table.table->size(0)), index, *rows))
        Py_RETURN_NONE;
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(index).stream();
    kda_status status;
    Py_BEGIN_ALLOW_THREADS
    status = resize_entry(table.refs->mutable_data_ptr<int32_t>(), table.n_pages,
                          table.table->mutable_data_ptr<int32_t>(), (int)table.table->size(0),
                          (int)table.table->size(1), rows->const_data_ptr<int32_t>(), tokens->const_data_ptr<int32_t>(),
                          (int)rows->numel(), page, missing.ptr(), ws.ptr(), ws.bytes(), stream);
    Py_END_ALLOW_THREADS
    if (failed(status)) return nullptr;
    return result(arg[5], missing.made);
    END_HANDLE_TH_ERRORS
}

// refs, block_table, lengths, src, dst, page, from_pages, to_pages, missing, workspace -> (from_pages, to_pages, missing)
PyObject* cache_fork(PyObject*, PyObject* const* arg, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    if (!takes("cache_fork", n_args, 10)) return nullptr;
    const at::Tensor *lengths = tensor(arg[2]), *src = tensor(arg[3]), *dst = tensor(arg[4]);
    const int index = current_device_of(src);
    Rows table;
    if (index < 0 || !table.read(arg[0], arg[1], index) || !dense(src, at::kInt, index) || src->dim() != 1 ||
        src->numel() > INT_MAX || !dense(dst, at::kInt, index, src->sizes()) ||
        !dense(lengths, at::kInt, index, {table.table->size(0)}))
        Py_RETURN_NONE;
    int page;
    if (!integer32(arg[5], page)) return nullptr;
    List from, to, missing;
    Workspace ws;
    if (!from.read(arg[6], src->numel(), index, *src) || !to.read(arg[7], src->numel(), index, *src) ||
        !missing.read(arg[8], 1, index, *src) || !ws.read(arg[9], pages_workspace_entry(table.n_pages, (int)table.table->size(0)), index, *src))
        Py_RETURN_NONE;
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(index).stream();
    kda_status status;
    Py_BEGIN_ALLOW_THREADS
    status = fork_entry(table.refs->mutable_data_ptr<int32_t>(), table.n_pages, table.table->mutable_data_ptr<int32_t>(),
                        (int)table.table->size(0), (int)table.table->size(1), lengths->mutable_data_ptr<int32_t>(),
                        src->const_data_ptr<int32_t>(), dst->const_data_ptr<int32_t>(), (int)src->numel(), page,
                        from.ptr(), to.ptr(), missing.ptr(), ws.ptr(), ws.bytes(), stream);
    Py_END_ALLOW_THREADS
    if (failed(status)) return nullptr;
    PyObject *a = result(arg[6], from.made), *b = result(arg[7], to.made), *c = result(arg[8], missing.made);
    PyObject* t = a && b && c ? PyTuple_Pack(3, a, b, c) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    Py_XDECREF(c);
    return t;
    END_HANDLE_TH_ERRORS
}

// refs, block_table, refs_out, table_out, page_map, from_pages, to_pages, held -> (page_map, from_pages, to_pages, held)
PyObject* cache_compact(PyObject*, PyObject* const* arg, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    if (!takes("cache_compact", n_args, 8)) return nullptr;
    const int index = current_device_of(tensor(arg[0]));
    Rows table;
    if (index < 0 || !table.read(arg[0], arg[1], index)) Py_RETURN_NONE;
    const at::Tensor *refs_out = table.refs, *table_out = table.table;
    if (arg[2] != Py_None && !dense(refs_out = tensor(arg[2]), at::kInt, index, table.refs->sizes())) Py_RETURN_NONE;
    if (arg[3] != Py_None && !dense(table_out = tensor(arg[3]), at::kInt, index, table.table->sizes())) Py_RETURN_NONE;
    List map, from, to, held;
    if (!map.read(arg[4], table.n_pages, index, *table.refs) || !from.read(arg[5], table.n_pages / 2, index, *table.refs) ||
        !to.read(arg[6], table.n_pages / 2, index, *table.refs) || !held.read(arg[7], 1, index, *table.refs))
        Py_RETURN_NONE;
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(index).stream();
    kda_status status;
    Py_BEGIN_ALLOW_THREADS
    status = compact_entry(table.refs->const_data_ptr<int32_t>(), refs_out->mutable_data_ptr<int32_t>(), table.n_pages,
                           table.table->const_data_ptr<int32_t>(), table_out->mutable_data_ptr<int32_t>(),
                           (int)table.table->size(0), (int)table.table->size(1), map.ptr(), from.ptr(), to.ptr(),
                           held.ptr(), stream);
    Py_END_ALLOW_THREADS
    if (failed(status)) return nullptr;
    PyObject* all[4] = {result(arg[4], map.made), result(arg[5], from.made), result(arg[6], to.made), result(arg[7], held.made)};
    PyObject* t = all[0] && all[1] && all[2] && all[3] ? PyTuple_Pack(4, all[0], all[1], all[2], all[3]) : nullptr;
    for (PyObject* x : all) Py_XDECREF(x);
    return t;
    END_HANDLE_TH_ERRORS
}

// q, cache, block_table, lengths, prefix_table, prefix_lengths, cu_groups, scale, out, lse, return_lse, workspace -> o or (o, lse)
PyObject* cache_attention_shared(PyObject*, PyObject* const* arg, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    if (!takes("cache_attention_shared", n_args, 12)) return nullptr;
    const at::Tensor *q = tensor(arg[0]), *table = tensor(arg[2]), *lengths = tensor(arg[3]);
    const at::Tensor *prefix = tensor(arg[4]), *prefix_len = tensor(arg[5]), *cu = tensor(arg[6]);
    const int index = current_device_of(q);
    kda_dtype code;
    if (index < 0 || !code_of(q->scalar_type(), code) || q->dim() != 4) Py_RETURN_NONE;
    const at::ScalarType type = q->scalar_type();
    const int64_t q_stride = token_stride(q, type, index);
    Pool pool;
    if (q_stride < 0 || !pool.read(arg[1], index) || q->size(3) != pool.d) Py_RETURN_NONE;
    const int64_t B = q->size(0), t_q = q->size(1), h_q = q->size(2);
    if (!dense(table, at::kInt, index) || table->dim() != 2 || table->size(0) != B || !dense(lengths, at::kInt, index, {B}) ||
        B > INT_MAX || t_q > INT_MAX || h_q > INT_MAX || table->size(1) > INT_MAX)
        Py_RETURN_NONE;
    if (!dense(prefix, at::kInt, index) || prefix->dim() != 2 || prefix->size(0) >= INT_MAX || prefix->size(1) > INT_MAX ||
        !dense(prefix_len, at::kInt, index, {prefix->size(0)}) || !dense(cu, at::kInt, index, {prefix->size(0) + 1}))
        Py_RETURN_NONE;
    const int wide = (int)table->size(1), d = (int)pool.d, groups = (int)prefix->size(0), prefix_wide = (int)prefix->size(1);
    float scale = (float)(1.0 / std::sqrt((double)d));
    if (arg[7] != Py_None && !real(arg[7], scale)) return nullptr;
    const int with_lse = PyObject_IsTrue(arg[10]);
    if (with_lse < 0) return nullptr;

    at::Tensor o_made, lse_made;
    const at::Tensor *o = &o_made, *lse = arg[9] != Py_None ? tensor(arg[9]) : with_lse ? &lse_made : nullptr;
    if (arg[8] != Py_None && !dense(o = tensor(arg[8]), type, index, q->sizes())) Py_RETURN_NONE;
    if (arg[9] != Py_None && !dense(lse, at::kFloat, index, q->sizes().slice(0, 3))) Py_RETURN_NONE;
    Workspace ws;
    const size_t need = arg[11] == Py_None ? shared_workspace_entry((int)B, (int)t_q, (int)h_q, (int)pool.h, d,
                                                                    (int)pool.page, wide, prefix_wide, groups)
                                           : 0;
    if (!ws.read(arg[11], need, index, *q)) Py_RETURN_NONE;
    if (arg[8] == Py_None) o_made = empty(q->sizes(), type, *q);
    if (lse == &lse_made) lse_made = empty(q->sizes().slice(0, 3), at::kFloat, *q);
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(index).stream();
    kda_status status;
    Py_BEGIN_ALLOW_THREADS
    status = shared_entry(q->const_data_ptr(), q_stride, pool.k->const_data_ptr(), pool.v->const_data_ptr(),
                          pool.k_scale->const_data_ptr<float>(), pool.v_scale->const_data_ptr<float>(),
                          table->const_data_ptr<int32_t>(), wide, lengths->const_data_ptr<int32_t>(),
                          prefix->const_data_ptr<int32_t>(), prefix_wide, prefix_len->const_data_ptr<int32_t>(),
                          cu->const_data_ptr<int32_t>(), groups, o->mutable_data_ptr(),
                          lse ? lse->mutable_data_ptr<float>() : nullptr, (int)B, (int)t_q, (int)h_q, (int)pool.h, d,
                          pool.n_pages, (int)pool.page, scale, code, ws.ptr(), ws.bytes(), stream);
    Py_END_ALLOW_THREADS
    if (failed(status)) return nullptr;
    PyObject* out = result(arg[8], o_made);
    return with_lse ? pair_of(out, result(arg[9], lse_made)) : out;
    END_HANDLE_TH_ERRORS
}

// The addresses of the entries, in the order of cache.py's list, and api._check
constexpr int kEntries = 12;
PyObject* bind(PyObject*, PyObject* const* arg, Py_ssize_t n_args) {
    if (!takes("bind", n_args, kEntries + 1)) return nullptr;
    void* at[kEntries];
    for (int i = 0; i < kEntries; ++i) {
        at[i] = PyLong_AsVoidPtr(arg[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    rotary_entry = reinterpret_cast<decltype(rotary_entry)>(at[0]);
    write_entry = reinterpret_cast<decltype(write_entry)>(at[1]);
    read_entry = reinterpret_cast<decltype(read_entry)>(at[2]);
    attention_entry = reinterpret_cast<decltype(attention_entry)>(at[3]);
    workspace_entry = reinterpret_cast<decltype(workspace_entry)>(at[4]);
    copy_entry = reinterpret_cast<decltype(copy_entry)>(at[5]);
    resize_entry = reinterpret_cast<decltype(resize_entry)>(at[6]);
    fork_entry = reinterpret_cast<decltype(fork_entry)>(at[7]);
    compact_entry = reinterpret_cast<decltype(compact_entry)>(at[8]);
    pages_workspace_entry = reinterpret_cast<decltype(pages_workspace_entry)>(at[9]);
    shared_entry = reinterpret_cast<decltype(shared_entry)>(at[10]);
    shared_workspace_entry = reinterpret_cast<decltype(shared_workspace_entry)>(at[11]);
    Py_XDECREF(check);
    check = Py_NewRef(arg[kEntries]);
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction method(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {{"bind", method(bind), METH_FASTCALL, nullptr},
                         {"rotary", method(rotary), METH_FASTCALL, nullptr},
                         {"cache_write", method(cache_write), METH_FASTCALL, nullptr},
                         {"cache_read", method(cache_read), METH_FASTCALL, nullptr},
                         {"cache_attention", method(cache_attention), METH_FASTCALL, nullptr},
                         {"cache_attention_shared", method(cache_attention_shared), METH_FASTCALL, nullptr},
                         {"cache_copy", method(cache_copy), METH_FASTCALL, nullptr},
                         {"cache_resize", method(cache_resize), METH_FASTCALL, nullptr},
                         {"cache_fork", method(cache_fork), METH_FASTCALL, nullptr},
                         {"cache_compact", method(cache_compact), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "kda_cache_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_kda_cache_binding() { return PyModule_Create(&module); }
